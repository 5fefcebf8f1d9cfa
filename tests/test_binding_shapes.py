"""The binding's checks of what the library cannot see: tensors whose sizes and types
do not belong together are refused before a pointer goes over. On the host: every call
here is refused, and none reaches a GPU."""
import pytest
import torch

import paged_kv_cache_154_gb300 as pa

KINDS = {"f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8,
         "fp8": torch.float8_e4m3fn, "int4": torch.uint8}
NB, H, D, T = 5, 3, 128, 4


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()


def cache(kv):
    width = D // 2 if kv == "int4" else D
    c = {n: torch.zeros((NB, H, 16, width), dtype=KINDS[kv]) for n in ("k_cache", "v_cache")}
    per = {"int8": (NB, H, 16), "int4": (NB, H, 16, D // 64), "fp8": (H,)}.get(kv)
    for n in ("k", "v"):
        c[n + "_scale"] = None if per is None else torch.zeros(per)
        c[n + "_zp"] = torch.zeros(per, dtype=torch.int8) if kv in ("int8", "int4") else None
    return c


def refuses(match, fn, **kw):
    """Refused by the binding, by the name of what is wrong."""
    with pytest.raises(ValueError, match=match):
        fn(**kw)


def scale_changes(kv):
    if kv == "int4":
        wrong = [torch.zeros((NB, H, 16)), torch.zeros((NB, H, 16, D // 64), dtype=torch.float64)]
        zps = [torch.zeros((NB, H, 16), dtype=torch.int8), torch.zeros((NB, H, 16, D // 64))]
    elif kv == "int8":
        wrong, zps = [torch.zeros((NB, H, 15))], [torch.zeros((NB, 1, 16), dtype=torch.int8)]
    elif kv == "fp8":
        wrong, zps = [torch.zeros(H - 1), torch.zeros(H, dtype=torch.float16)], []
    else:
        wrong, zps = [], []
    return [(n + "_scale", t) for n in "kv" for t in wrong] + [(n + "_zp", t) for n in "kv"
                                                              for t in zps]


@pytest.mark.parametrize("kv", KINDS)
def test_gather(kv):
    def args():
        return dict(key=torch.zeros((T, H, D)), value=torch.zeros((T, H, D)), **cache(kv),
                    slot_mapping=torch.full((T,), -1))
    for value in (torch.zeros((T - 1, H, D)), torch.zeros((T, H, D // 2)), torch.zeros((T, H + 1, D)),
                  torch.zeros((T, H, D), dtype=torch.float16)):
        refuses("value", pa.gather_kv, **{**args(), "value": value})
    refuses("key", pa.gather_kv, **{**args(), "key": torch.zeros((T, H * D // 2))})
    for slots in (torch.zeros(T, dtype=torch.int32), torch.zeros(T - 1, dtype=torch.int64)):
        refuses("slot_mapping", pa.gather_kv, **{**args(), "slot_mapping": slots})
    refuses("num_blocks", pa.gather_kv, **args(), num_blocks=NB + 1)
    refuses("v_cache", pa.gather_kv, **{**args(), "v_cache": torch.zeros_like(cache(kv)["k_cache"])[:2]})
    for name, t in scale_changes(kv):
        refuses(name, pa.gather_kv, **{**args(), name: t})


def test_append_and_copy_of_an_int4_cache():
    def args():
        return dict(key=torch.zeros((T, H, D), dtype=torch.float16), **cache("int4"),
                    value=torch.zeros((T, H, D), dtype=torch.float16),
                    slot_mapping=torch.full((T,), -1))
    refuses("value", pa.append_kv, **{**args(), "value": torch.zeros((T, H, D - 1)).half()})
    refuses("value", pa.append_kv, **{**args(), "value": torch.zeros((T, H, D)).bfloat16()})
    refuses("slot_mapping", pa.append_kv, **{**args(), "slot_mapping": torch.zeros(T).int()})
    pairs = torch.zeros((1, 2), dtype=torch.int32)
    for name, t in scale_changes("int4"):
        refuses(name, pa.append_kv, **{**args(), name: t})
        refuses(name, pa.copy_blocks, **{**cache("int4"), name: t}, pairs=pairs)
    for call, kw in ((pa.append_kv, args()), (pa.copy_blocks, dict(cache("int4"), pairs=pairs))):
        refuses("num_blocks", call, **kw, num_blocks=NB + 1)


@pytest.mark.parametrize("call", [pa.decode, pa.decode_no_alloc], ids=lambda f: f.__name__)
def test_decode_of_an_int4_cache(call):
    def args():
        q = torch.zeros((1, 2 * H, D), dtype=torch.float16)
        return dict(out=torch.zeros(q.shape), q=q, **cache("int4"), max_context_len=16, scale=1.0,
                    block_tables=torch.zeros((1, 1), dtype=torch.int32),
                    context_lens=torch.ones(1, dtype=torch.int32))
    refuses("head_dim", call, **{**args(), "q": torch.zeros((1, 2 * H, 2 * D)).half()})
    refuses("out", call, **{**args(), "out": torch.zeros((1, H, D))})
    refuses("num_blocks", call, **args(), num_blocks=NB + 1)
    for name, t in scale_changes("int4"):
        refuses(name, call, **{**args(), name: t})


@pytest.mark.parametrize("kv", KINDS)
def test_weights_and_moves(kv):
    c = cache(kv)
    lens, bt = torch.ones(1, dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32)
    w = dict(scores_out=torch.zeros((1, H, 16)), scores_in=None, q=torch.zeros((1, 2 * H, D)).half(),
             k_cache=c["k_cache"], block_tables=bt, context_lens=lens, max_context_len=16, scale=1.0,
             k_scale=c["k_scale"], k_zp=c["k_zp"])
    m = dict(c, block_tables=bt, context_lens=lens, max_context_len=16,
             moves=torch.zeros((1, H, 8, 2), dtype=torch.int32),
             move_counts=torch.zeros((1, H), dtype=torch.int32))
    refuses("head_dim", pa.accumulate_weights, **{**w, "q": torch.zeros((1, 2 * H, 2 * D)).half()})
    refuses("v_cache", pa.move_tokens, **{**m, "v_cache": c["v_cache"][:NB - 1]})
    for call, kw in ((pa.accumulate_weights, w), (pa.move_tokens, m)):
        refuses("num_blocks", call, **kw, num_blocks=NB + 1)
        for name, t in scale_changes(kv):
            if name in kw:
                refuses(name, call, **{**kw, name: t})
