// The calls with their arguments in one array (see pa.h): for bindings that convert
// arguments one by one.
#include <string.h>

#include <initializer_list>

#include "pa_internal.h"

namespace {

template <typename T>
T* at(int64_t word) {
    return reinterpret_cast<T*>(static_cast<uintptr_t>(word));
}
int32_t i32(int64_t word) { return static_cast<int32_t>(word); }
pa_dtype type(int64_t word) { return static_cast<pa_dtype>(word); }
// The array is there, and what the call takes as 32 bits (words whose places are given) fits them.
pa_status check(const int64_t* a, std::initializer_list<int> small) {
    if (!a) return pa::fail(PA_ERR_INVALID_ARG, "args is NULL");
    for (int i : small)
        if (a[i] != static_cast<int32_t>(a[i]))
            return pa::fail(PA_ERR_INVALID_ARG, "argument %d, %lld, is no 32-bit number", i,
                            (long long)a[i]);
    return PA_OK;
}

}  // namespace

extern "C" pa_status pa_rope_packed(const int64_t* a) {
    if (pa_status s = check(a, {4, 9, 10, 12, 13, 14, 16, 18, 19, 20})) return s;
    return pa_rope(at<void>(a[0]), a[1], at<const void>(a[2]), a[3], i32(a[4]), at<void>(a[5]), a[6],
                   at<const void>(a[7]), a[8], i32(a[9]), type(a[10]), at<const float>(a[11]),
                   i32(a[12]), i32(a[13]), i32(a[14]), at<const int32_t>(a[15]), i32(a[16]),
                   at<const uint8_t>(a[17]), i32(a[18]), i32(a[19]), i32(a[20]), at<void>(a[21]));
}

extern "C" pa_status pa_rope_append_kv_packed(const int64_t* a) {
    if (pa_status s = check(a, {4, 11, 14, 21, 22, 23, 25, 27, 28, 29, 30, 31})) return s;
    return pa_rope_append_kv(
        at<void>(a[0]), a[1], at<const void>(a[2]), a[3], i32(a[4]), at<void>(a[5]), a[6],
        at<const void>(a[7]), a[8], at<const void>(a[9]), a[10], type(a[11]), at<void>(a[12]),
        at<void>(a[13]), type(a[14]), at<float>(a[15]), at<float>(a[16]), at<int8_t>(a[17]),
        at<int8_t>(a[18]), at<const int64_t>(a[19]), at<const float>(a[20]), i32(a[21]), i32(a[22]),
        i32(a[23]), at<const int32_t>(a[24]), i32(a[25]), at<const uint8_t>(a[26]), i32(a[27]),
        i32(a[28]), i32(a[29]), i32(a[30]), i32(a[31]), at<void>(a[32]));
}

extern "C" pa_status pa_prompt_attention_packed(const int64_t* a) {
    if (pa_status s = check(a, {8, 10, 11, 12, 13, 14, 15})) return s;
    double scale;
    memcpy(&scale, a + 16, sizeof scale);
    return pa_prompt_attention(at<void>(a[0]), a[1], at<const void>(a[2]), a[3],
                               at<const void>(a[4]), a[5], at<const void>(a[6]), a[7], type(a[8]),
                               at<const int32_t>(a[9]), i32(a[10]), i32(a[11]), i32(a[12]),
                               i32(a[13]), i32(a[14]), i32(a[15]), static_cast<float>(scale),
                               at<void>(a[17]), static_cast<size_t>(a[18]), at<void>(a[19]));
}
