"""Refusals of the paged operators: what can be refused without a GPU."""

import ctypes

import pytest
import torch

from conftest import build_lib


@pytest.fixture(scope="module")
def tq():
    return build_lib()


def structs(tq, **kw):
    """Arguments that would be accepted but for the missing handles (addresses are never followed by the host)."""
    p = 1 << 12
    v = {"codes": p, "signs": p, "norms": p, "rnorms": p, "num_pages": 4, "page_size": 16,
         "q_start": p, "len": p, "block_table": p, "B": 2, "max_pages": 2, "ntok": 3, "max_q": 2,
         "cos_sin": p, "pos": p, "weight": p, "max_pos": 16, "rot_dim": 64, "interleaved": 0, "weight_dtype": 0, "eps": 1e-6,
         "Hkv": 2, "Hq": 4, "dtype": tq.TQ_BF16, "scale": 0.1, "causal": 1, "window": 0}
    v.update(kw)
    cache = tq._lib.tq_paged_cache(*(v[k] for k in ("codes", "signs", "norms", "rnorms", "num_pages", "page_size")))
    batch = tq._lib.tq_paged_batch(*(v[k] for k in ("q_start", "len", "block_table", "B", "max_pages", "ntok", "max_q")))
    prep = tq._lib.tq_head_prep(*(v[k] for k in ("cos_sin", "pos", "weight", "max_pos", "rot_dim", "interleaved",
                                                 "weight_dtype", "eps")))
    return v, cache, batch, prep


def refuse(tq, kw, word, which=("append", "attn")):
    v, cache, batch, prep = structs(tq, **{k: x for k, x in kw.items() if not k.startswith("no_")})
    r = ctypes.byref
    other = tq._lib.tq_paged_cache(1 << 12, 1 << 12, 1 << 12, 1 << 12, v["num_pages"], kw.get("no_v_page", v["page_size"]))
    b = None if kw.get("no_batch") else r(batch)
    c = None if kw.get("no_cache") else r(cache)
    if "append" in which:
        st = tq._lib.lib.tq_append_paged(None, None, 4096, 4096, v["dtype"], 4096, 4096, v["Hkv"], b, r(prep), c, r(other), None)
        assert st == tq.TQ_EINVAL and word in tq.tq_last_error(), tq.tq_last_error()
    if "attn" in which:
        st = tq._lib.lib.tq_attn_paged(None, None, 4096, v["dtype"], 4096, v["Hq"], v["Hkv"], b, r(prep), c, r(other),
                                       v["scale"], v["causal"], v["window"], 4096, 4096, 1 << 20, None)
        assert st == tq.TQ_EINVAL and word in tq.tq_last_error(), tq.tq_last_error()


BOTH = [
    ({}, "handle is NULL"), ({"no_batch": True}, "batch is NULL"), ({"no_cache": True}, "cache is NULL"),
    ({"page_size": 8}, "page_size"), ({"page_size": 24}, "page_size"), ({"page_size": 2048}, "page_size"),
    ({"no_v_page": 32}, "block table"), ({"num_pages": 0}, "num_pages"), ({"norms": 0}, "norms"),
    ({"codes": 4100}, "alignment"), ({"rnorms": 4098}, "alignment"),
    ({"B": -1}, "B="), ({"B": 1 << 20}, "B="), ({"ntok": -1}, "ntok"), ({"ntok": 1 << 25}, "ntok"),
    ({"max_pages": 0}, "max_pages"), ({"max_pages": 1 << 27}, "max_pages"), ({"max_q": 4}, "max_q"), ({"max_q": -1}, "max_q"),
    ({"q_start": 0}, "NULL"), ({"len": 0}, "NULL"), ({"block_table": 0}, "NULL"), ({"len": 4098}, "misaligned"),
    ({"rot_dim": 4}, "rot_dim"), ({"rot_dim": 68}, "rot_dim"), ({"max_pos": 0}, "max_pos"), ({"interleaved": 2}, "interleaved"),
    ({"cos_sin": 4100}, "misaligned"), ({"pos": 4098}, "misaligned"), ({"eps": 0.0}, "eps"), ({"eps": float("inf")}, "eps"),
    ({"weight_dtype": 7}, "weight dtype"), ({"dtype": 9}, "dtype"), ({"Hkv": 0}, "Hkv"), ({"Hkv": 4096}, "Hkv"),
]


@pytest.mark.parametrize("kw,word", BOTH)
def test_refusals_of_both(tq, kw, word):
    refuse(tq, kw, word)


@pytest.mark.parametrize("kw,word", [
    ({"Hq": 3}, "Hq"), ({"Hq": 0}, "Hq"), ({"Hq": 2048}, "Hq"), ({"scale": float("nan")}, "scale"), ({"causal": 2}, "causal"),
    ({"window": -1}, "window"), ({"window": 5, "causal": 0}, "window"), ({"causal": 0, "pos": 0}, "prep->pos")])
def test_refusals_of_attention(tq, kw, word):
    refuse(tq, kw, word, ("attn",))


def test_workspace_size_of_a_refused_call_is_zero(tq):
    v, cache, batch, prep = structs(tq)
    assert tq.tq_attn_paged_workspace_bytes(None, None, batch, 4, 2, cache) == 0


def test_binding_refuses_host_tensors_and_shapes(tq):
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(tq.TQError):
        tq.PagedBatch(i, i[:2], torch.zeros(2, 2, dtype=torch.int32), 3)
    with pytest.raises(tq.TQError):
        tq.HeadPrep(cos_sin=torch.zeros(4, 64))
    with pytest.raises(tq.TQError):
        tq.HeadPrep(weight=torch.zeros(64))


def test_binding_refuses_other_devices(tq):
    """A handle, a cache, a batch or a stream of another device would have a kernel follow addresses that are not its own."""
    from types import SimpleNamespace as obj
    mod = tq

    def things(**at):
        h = [obj(d=128, bits_mse=4, m=0, norm_dtype=1, index=at.get(n, 0)) for n in ("hk", "hv")]
        c = [obj(handle=h[i], Hkv=2, index=at.get(n, 0)) for i, n in enumerate(("kcache", "vcache"))]
        return (*h, *c, obj(index=at.get("batch", 0), ntok=1), obj(index=at.get("prep", 0), weight=None, pos=None))

    mod._check_paged(*things())
    for name in ("hk", "hv", "kcache", "vcache", "batch", "prep"):
        with pytest.raises(tq.TQError, match="device"):
            mod._check_paged(*things(**{name: 1}))
    with pytest.raises(tq.TQError, match="device"):
        mod._on(obj(device_index=1), torch.device("cuda", 0))
