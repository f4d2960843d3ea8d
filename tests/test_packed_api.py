"""Host side of the packed operators (no GPU): exported symbols, the plan, refused arguments, and
the reference the GPU tests compare with."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import packed_ref as R
from fwd_bwd_b200 import _lib, packed, rope
from fwd_bwd_b200._lib import SagePackedInfo, SagePackedParams, SageRopeParams, SageRows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # a device address that no call below reaches: each fails its host-side checks


@pytest.fixture(scope="module")
def L():
    import fwd_bwd_b200.build as b

    b.build()
    return _lib.lib()


def test_exports(L):
    src = open(os.path.join(ROOT, "include", "sage_packed.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(sage_[a-z0-9_]+)\s*\(", src)))
    assert names == ["sage_packed_attn_bwd", "sage_packed_attn_bwd_workspace_bytes",
                     "sage_packed_attn_fwd", "sage_packed_attn_fwd_workspace_bytes",
                     "sage_packed_plan_bytes", "sage_packed_plan_fill",
                     "sage_qk_norm_rope_bwd", "sage_qk_norm_rope_fwd",
                     "sage_qk_norm_rope_workspace_bytes"]
    for n in names:
        assert hasattr(L, n), n


@pytest.mark.parametrize("lengths", [[1], [0], [0, 0, 7], [128], [129, 1, 256], [300, 0, 5, 1024],
                                     list(range(40)), [65537, 3]])
def test_plan(L, lengths):
    b = packed.Batch(lengths, device="cpu")
    info = b.info
    tiles = [-(-n // 128) for n in lengths]
    assert info.sequences == len(lengths) and info.tokens == sum(lengths) == b.tokens
    assert info.tiles == sum(tiles) and info.longest == max(lengths)
    assert info.pairs == sum((t + 1) // 2 for t in tiles)
    assert info.causal_steps == sum(t * (t + 1) // 2 for t in tiles)
    assert info.full_steps == sum(t * t for t in tiles)
    items = b.plan.numpy().view(np.int32).reshape(-1, 4)
    assert len(items) == 2 * (info.tiles + info.pairs) + 1  # never empty
    starts = np.concatenate([[0], np.cumsum(lengths)])
    at = 0
    for count, step, causal in ((info.tiles, 1, True), (info.tiles, 1, False),
                                (info.pairs, 2, True), (info.pairs, 2, False)):
        part = items[at:at + count]
        at += count
        want = {(s, t) for s, n in enumerate(tiles) for t in range(n - 1, -1, -step)}
        assert {(s, t) for _, _, t, s in part.tolist()} == want and len(part) == len(want)
        assert all(start == starts[s] and n == lengths[s] for start, n, _, s in part.tolist())
        work = [t + 1 if causal else tiles[s] for _, _, t, s in part.tolist()]
        assert work == sorted(work, reverse=True)
    if sum(lengths):
        pos = b.positions()
        assert pos.dtype == torch.int32
        assert pos.tolist() == [i for n in lengths for i in range(n)]


def test_plan_refusals(L):
    for bad in ([], [-1], [5, -2], [2 ** 31], [2 ** 30, 2 ** 30], [1 << 30, (1 << 30) - 128]):
        with pytest.raises((ValueError, _lib.SageError)):
            packed.Batch(bad, device="cpu")
    for bad in (torch.ones(3), torch.ones((2, 2), dtype=torch.int64)):
        with pytest.raises(ValueError):
            packed.Batch(bad, device="cpu")
    assert packed.Batch(torch.tensor([3, 4]), device="cpu").lengths == [3, 4]
    arr = (ctypes.c_int * 2)(5, 200)
    info = SagePackedInfo()
    n = L.sage_packed_plan_bytes(arr, 2)
    buf = ctypes.create_string_buffer(n)
    fill = L.sage_packed_plan_fill
    assert fill(arr, 2, buf, n, ctypes.byref(info)) == _lib.SAGE_OK
    assert fill(arr, 2, buf, n - 1, ctypes.byref(info)) == _lib.SAGE_ERR_WORKSPACE
    assert fill(arr, 2, None, n, ctypes.byref(info)) == _lib.SAGE_ERR_INVALID_ARG
    assert fill(arr, 2, buf, n, None) == _lib.SAGE_ERR_INVALID_ARG
    assert fill(arr, 0, buf, n, ctypes.byref(info)) == _lib.SAGE_ERR_INVALID_ARG
    assert L.sage_packed_plan_bytes(None, 2) == 0


def _info(lengths=(100, 28)):
    return packed.Batch(list(lengths), device="cpu").info


def _rows(heads, d=64, T=128, ptr=FAKE, **kw):
    f = dict(ptr=ptr, batch_stride=0, token_stride=heads * d, head_stride=d)
    f.update(kw)
    return SageRows(*f.values())


def test_attention_refusals(L):
    info = _info()
    good = dict(T=128, Hq=4, Hkv=2, d=64, dtype=1, causal=1, softmax_scale=0.0)

    def fwd(prm=None, inf=info, plan=FAKE, lse=FAKE, **rows):
        p = SagePackedParams(*{**good, **(prm or {})}.values())
        r = {"q": _rows(4), "k": _rows(2), "v": _rows(2), "o": _rows(4), **rows}
        return L.sage_packed_attn_fwd(ctypes.byref(p), ctypes.byref(inf), plan, *r.values(), lse,
                                      None, 0, None)

    E = _lib
    for prm, code in ((dict(d=96), E.SAGE_ERR_UNSUPPORTED), (dict(d=256), E.SAGE_ERR_UNSUPPORTED),
                      (dict(Hq=5), E.SAGE_ERR_INVALID_ARG), (dict(Hkv=0), E.SAGE_ERR_INVALID_ARG),
                      (dict(T=0), E.SAGE_ERR_INVALID_ARG), (dict(T=127), E.SAGE_ERR_INVALID_ARG),
                      (dict(T=1 << 31), E.SAGE_ERR_UNSUPPORTED), (dict(dtype=2), E.SAGE_ERR_INVALID_ARG),
                      (dict(causal=2), E.SAGE_ERR_INVALID_ARG),
                      (dict(softmax_scale=math.nan), E.SAGE_ERR_INVALID_ARG)):
        assert fwd(prm) == code, prm
    assert fwd(plan=None) == E.SAGE_ERR_INVALID_ARG
    assert fwd(plan=FAKE + 8) == E.SAGE_ERR_ALIGNMENT
    assert fwd(lse=None) == E.SAGE_ERR_INVALID_ARG
    assert fwd(q=_rows(4, ptr=None)) == E.SAGE_ERR_INVALID_ARG
    assert fwd(k=_rows(2, ptr=FAKE + 2)) == E.SAGE_ERR_ALIGNMENT
    assert fwd(v=_rows(2, token_stride=132)) == E.SAGE_ERR_ALIGNMENT
    assert fwd(k=_rows(2, head_stride=0)) == E.SAGE_ERR_INVALID_ARG
    assert fwd(q=_rows(4, token_stride=-256)) == E.SAGE_ERR_INVALID_ARG
    assert fwd(q=_rows(4, token_stride=1 << 40)) == E.SAGE_ERR_INVALID_ARG
    assert fwd(o=_rows(4, token_stride=64)) == E.SAGE_ERR_INVALID_ARG  # vectors overlap
    assert fwd(o=_rows(4, token_stride=192)) == E.SAGE_ERR_INVALID_ARG
    bad = SagePackedInfo(2, 2, 3, 100, 128)
    assert fwd(inf=bad) == E.SAGE_ERR_INVALID_ARG
    # nothing to do is not an error
    empty = SagePackedInfo(2, 0, 0, 0, 0)
    assert fwd(inf=empty) == E.SAGE_OK

    # few heads and a long sequence: parts, which need a workspace
    p = SagePackedParams(*good.values())
    need = L.sage_packed_attn_fwd_workspace_bytes
    assert need(ctypes.byref(p), ctypes.byref(info)) == 0
    long = _info([128 * 100])
    pl = SagePackedParams(*{**good, "T": 12800}.values())
    n = need(ctypes.byref(pl), ctypes.byref(long))
    assert n >= 2 * 12800 * 4 * (64 + 2) * 4
    args = (ctypes.byref(pl), ctypes.byref(long), FAKE, _rows(4), _rows(2), _rows(2), _rows(4), FAKE)
    assert L.sage_packed_attn_fwd(*args, None, 0, None) == E.SAGE_ERR_WORKSPACE
    assert L.sage_packed_attn_fwd(*args, FAKE, n - 1, None) == E.SAGE_ERR_WORKSPACE
    assert L.sage_packed_attn_fwd(*args, FAKE + 8, n, None) == E.SAGE_ERR_ALIGNMENT

    ws = L.sage_packed_attn_bwd_workspace_bytes(ctypes.byref(p), ctypes.byref(info))
    assert ws == 4 * 128 * 4
    half = SagePackedParams(*{**good, "dtype": 0}.values())
    assert L.sage_packed_attn_bwd_workspace_bytes(ctypes.byref(half), ctypes.byref(info)) > ws
    wrong = SagePackedParams(*{**good, "d": 96}.values())
    assert L.sage_packed_attn_bwd_workspace_bytes(ctypes.byref(wrong), ctypes.byref(info)) == 0

    def bwd(w=FAKE, n=ws, lse=FAKE, prm=p, **rows):
        r = {"q": _rows(4), "k": _rows(2), "v": _rows(2), "o": _rows(4), **rows}
        s = {"dout": _rows(4), "dq": _rows(4), "dk": _rows(2), "dv": _rows(2)}
        for name in s:
            s[name] = r.pop(name, s[name])
        return L.sage_packed_attn_bwd(ctypes.byref(prm), ctypes.byref(info), FAKE, *r.values(), lse,
                                      *s.values(), w, n, None)

    assert bwd(prm=wrong) == E.SAGE_ERR_UNSUPPORTED
    assert bwd(w=None) == E.SAGE_ERR_WORKSPACE
    assert bwd(n=ws - 1) == E.SAGE_ERR_WORKSPACE
    assert bwd(w=FAKE + 4) == E.SAGE_ERR_ALIGNMENT
    assert bwd(lse=None) == E.SAGE_ERR_INVALID_ARG
    assert bwd(dk=_rows(2, token_stride=64)) == E.SAGE_ERR_INVALID_ARG
    assert bwd(dout=_rows(4, ptr=FAKE + 8)) == E.SAGE_ERR_ALIGNMENT
    assert bwd(dq=_rows(4, ptr=None)) == E.SAGE_ERR_INVALID_ARG


def test_rope_refusals(L):
    freq = (ctypes.c_double * 32)(*[1.0] * 32)
    good = dict(B=1, N=10, Hq=2, Hkv=1, d=64, dtype=1, norm=1, eps=1e-6, rotary_dim=64,
                interleaved=0, n_axes=1, sections=(32, 0, 0, 0), inv_freq=freq, pos_bits=32,
                pos_axis_stride=10, pos_batch_stride=0)

    def params(**kw):
        f = {**good, **kw}
        f["sections"] = (ctypes.c_int * 4)(*f["sections"])
        f["inv_freq"] = ctypes.cast(f["inv_freq"], ctypes.c_void_p) if f["inv_freq"] else None
        return SageRopeParams(*f.values())

    def fwd(pos=FAKE, gain=FAKE, rows=None, **kw):
        r = {"q": _rows(2), "k": _rows(1), "yq": _rows(2), "yk": _rows(1), **(rows or {})}
        r = list(r.values())
        return L.sage_qk_norm_rope_fwd(ctypes.byref(params(**kw)), r[0], r[1], gain, gain, pos, r[2],
                                       r[3], None)

    E = _lib
    for kw, code in ((dict(d=96), E.SAGE_ERR_UNSUPPORTED), (dict(N=0), E.SAGE_ERR_INVALID_ARG),
                     (dict(B=1 << 16, N=1 << 16), E.SAGE_ERR_UNSUPPORTED),
                     (dict(dtype=5), E.SAGE_ERR_INVALID_ARG), (dict(eps=-1.0), E.SAGE_ERR_INVALID_ARG),
                     (dict(eps=math.nan), E.SAGE_ERR_INVALID_ARG),
                     (dict(rotary_dim=8), E.SAGE_ERR_UNSUPPORTED),
                     (dict(rotary_dim=80), E.SAGE_ERR_INVALID_ARG),
                     (dict(rotary_dim=-16), E.SAGE_ERR_INVALID_ARG),
                     (dict(n_axes=0), E.SAGE_ERR_INVALID_ARG), (dict(n_axes=5), E.SAGE_ERR_INVALID_ARG),
                     (dict(sections=(31, 0, 0, 0)), E.SAGE_ERR_INVALID_ARG),
                     (dict(n_axes=2, sections=(32, 0, 0, 0)), E.SAGE_ERR_INVALID_ARG),
                     (dict(inv_freq=(ctypes.c_double * 32)(*[math.inf] * 32)), E.SAGE_ERR_INVALID_ARG),
                     (dict(inv_freq=None), E.SAGE_ERR_INVALID_ARG),
                     (dict(pos_bits=16), E.SAGE_ERR_INVALID_ARG), (dict(norm=2), E.SAGE_ERR_INVALID_ARG),
                     (dict(interleaved=3), E.SAGE_ERR_INVALID_ARG),
                     (dict(pos_axis_stride=-1), E.SAGE_ERR_INVALID_ARG)):
        assert fwd(**kw) == code, kw
    assert fwd(pos=None) == E.SAGE_ERR_INVALID_ARG
    assert fwd(norm=0) == E.SAGE_ERR_INVALID_ARG  # gains without a norm
    assert fwd(rows={"q": _rows(2, ptr=FAKE + 4)}) == E.SAGE_ERR_ALIGNMENT
    assert fwd(rows={"yq": _rows(2, token_stride=64)}) == E.SAGE_ERR_INVALID_ARG
    assert fwd(rows={"yk": _rows(1, ptr=None)}) == E.SAGE_ERR_INVALID_ARG
    ws = L.sage_qk_norm_rope_workspace_bytes(ctypes.byref(params()))
    assert ws > 0
    assert L.sage_qk_norm_rope_workspace_bytes(ctypes.byref(params(d=32))) == 0

    def bwd(dgq=FAKE, dgk=FAKE, w=FAKE, n=ws, gain=FAKE, **kw):
        r = [_rows(2), _rows(1)]
        return L.sage_qk_norm_rope_bwd(ctypes.byref(params(**kw)), *r, gain, gain, FAKE, *r, *r, dgq,
                                       dgk, w, n, None)

    assert bwd(dgk=None) == E.SAGE_ERR_INVALID_ARG
    assert bwd(w=None) == E.SAGE_ERR_WORKSPACE
    assert bwd(n=ws - 1) == E.SAGE_ERR_WORKSPACE
    assert bwd(w=FAKE + 8) == E.SAGE_ERR_ALIGNMENT
    assert bwd(norm=0, gain=None) == E.SAGE_ERR_INVALID_ARG  # gradients of gains without a norm


def test_rope_object_refusals():
    for kw in (dict(d=96), dict(d=64, rotary_dim=24), dict(d=64, rotary_dim=80),
               dict(d=64, sections=[16, 15]), dict(d=64, sections=[32, 0]),
               dict(d=128, sections=[16, 16, 16, 8, 8]), dict(d=64, inv_freq=[1.0] * 31),
               dict(d=64, inv_freq=[math.nan] * 32), dict(d=64, base=0.0), dict(d=64, eps=-1.0)):
        with pytest.raises(ValueError):
            rope.Rope(**kw)
    assert rope.Rope(64).axes == 1 and rope.Rope(64, rotary_dim=0).axes == 0


def test_cpu_tensors_are_refused():
    q, k = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros((4, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        packed.attn_fwd(q, k, k, packed.Batch([4], device="cpu"))
    with pytest.raises(ValueError, match="CUDA"):
        rope.qk_norm_rope_fwd(q, k, torch.arange(4), rope.Rope(64))


# ---- the reference itself ------------------------------------------------------------------
def test_reference_attention_against_differences():
    torch.manual_seed(0)
    lengths, hq, hkv, d = [5, 0, 3], 4, 2, 8
    q, k, v, do = (torch.randn((8, h, d), dtype=torch.float64) for h in (hq, hkv, hkv, hq))
    for causal in (True, False):
        ref = R.attention(q, k, v, lengths, causal, 0.3, do)
        # against a direct evaluation, row by row
        at = 0
        for n in lengths:
            for h in range(hq):
                for i in range(n):
                    m = i + 1 if causal else n
                    z = (k[at:at + m, h // 2] @ q[at + i, h]) * 0.3
                    w = z.exp() / z.exp().sum()
                    assert torch.allclose(ref["o"][at + i, h], w @ v[at:at + m, h // 2])
                    assert torch.allclose(ref["lse"][h, at + i], z.exp().sum().log())
            at += n

        def loss():
            return float((R.attention(q, k, v, lengths, causal, 0.3)["o"] * do).sum())

        for name, x in (("dq", q), ("dk", k), ("dv", v)):
            for idx in ((0, 0, 0), (4, 1, 3), (7, 0, 7), (2, 1, 5)):
                old = x[idx].item()
                x[idx] = old + 1e-5
                up = loss()
                x[idx] = old - 1e-5
                down = loss()
                x[idx] = old
                assert abs((up - down) / 2e-5 - float(ref[name][idx])) < 1e-8, (name, idx)


def test_reference_rope_against_differences():
    torch.manual_seed(1)
    T, H, d = 3, 2, 8
    x, dy = (torch.randn((T, H, d), dtype=torch.float64) for _ in range(2))
    gain = torch.rand(d, dtype=torch.float64) + 0.5
    pos = torch.tensor([[0, 7, 100], [3, 2, 1]])
    for inter in (False, True):
        for norm in (True, False):
            g = gain if norm else None
            args = (pos, [1.0, 0.3, 0.01], [2, 1], inter, norm, 1e-3)
            ref = R.rope(x, g, *args, dy)
            # a rotation keeps every pair's length
            y = ref["y"]
            z = x / (x.pow(2).mean(-1, keepdim=True) + 1e-3).sqrt() * gain if norm else x
            assert torch.allclose(y.pow(2).sum(-1), z.pow(2).sum(-1))
            lo, hi = (0, 1) if inter else (0, 3)
            a, b = z[1, 0, lo], z[1, 0, hi]
            assert torch.allclose(y[1, 0, lo], a * math.cos(7.0) - b * math.sin(7.0))
            for idx in ((0, 0, 0), (1, 1, 4), (2, 0, 7)):
                old = x[idx].item()
                x[idx] = old + 1e-5
                up = float((R.rope(x, g, *args)["y"] * dy).sum())
                x[idx] = old - 1e-5
                down = float((R.rope(x, g, *args)["y"] * dy).sum())
                x[idx] = old
                assert abs((up - down) / 2e-5 - float(ref["dx"][idx])) < 1e-8
            if norm:
                old = gain[2].item()
                gain[2] = old + 1e-5
                up = float((R.rope(x, gain, *args)["y"] * dy).sum())
                gain[2] = old - 1e-5
                down = float((R.rope(x, gain, *args)["y"] * dy).sum())
                gain[2] = old
                assert abs((up - down) / 2e-5 - float(ref["dgain"][2])) < 1e-8
