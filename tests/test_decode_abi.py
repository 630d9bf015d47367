"""Refusals of the decode cycle's calls, and the frequencies of rotary positions (CPU only:
arguments are checked on the host and the placeholder pointers are never followed)."""
import ctypes

import numpy as np
import pytest

from speculative_decoding_tree_04_gb300 import tv
from tests import decode_model as dm

FAKE, M = 1 << 30, 1 << 20
BAD, UNS = tv.TV_ERR_INVALID_ARG, tv.TV_ERR_UNSUPPORTED


def fill(a, kw):
    a.struct_size = ctypes.sizeof(a)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def rope_args(**kw):
    a = tv.RopeArgs()
    a.T, a.n_heads, a.d_head, a.rot_offset, a.rot_dim = 10, 4, 64, 16, 48
    a.dt, a.in_, a.out, a.positions = tv.TV_F32, FAKE, FAKE + M, FAKE + 2 * M
    a.in_stride_token, a.in_stride_head = a.out_stride_token, a.out_stride_head = 256, 64
    a.scaling = tv.rope_scaling()
    return fill(a, kw)


SCALINGS = [
    (dict(base=1.0), BAD), (dict(base=float("inf")), BAD), (dict(base=float("nan")), BAD),
    (dict(kind=5), BAD), (dict(kind=-1), BAD), (dict(kind=1, factor=0.5), BAD),
    (dict(kind=2, factor=float("nan")), BAD), (dict(kind=3, factor=2, original_context=0), BAD),
    (dict(kind=3, factor=2, low=5, high=5), BAD), (dict(kind=4, factor=2, low=0), BAD),
    (dict(magnitude=float("inf")), BAD), (dict(kind=0, factor=0.5), tv.TV_OK),
]


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=8), BAD), (dict(T=-1), BAD), (dict(n_heads=0), BAD), (dict(d_head=1), BAD),
    (dict(rot_offset=-1), BAD), (dict(rot_dim=0), BAD), (dict(rot_dim=47), BAD),
    (dict(rot_dim=514, d_head=600), BAD), (dict(rot_dim=50), BAD), (dict(d_head=65537), UNS),
    (dict(layout=2), BAD), (dict(inverse=2), BAD), (dict(dt=2), BAD), (dict(in_=None), BAD),
    (dict(positions=None), BAD), (dict(out=FAKE + M + 2), BAD), (dict(out_stride_head=63), BAD),
    (dict(out_stride_token=255), BAD), (dict(in_stride_token=-1), BAD),
    (dict(in_stride_head=1 << 31), BAD), (dict(out=FAKE, out_stride_token=512), BAD),
    (dict(positions=FAKE + M + 4 * (9 * 256 + 255)), BAD), (dict(T=0, in_=None), tv.TV_OK),
])
def test_rope_arguments(tvlib, kw, code):
    assert tv.load().tv_rope(ctypes.byref(rope_args(**kw)), None) == code
    assert (code == tv.TV_OK) == (not tv.load().tv_last_error())


@pytest.mark.parametrize("kw,code", SCALINGS)
def test_scaling_arguments(tvlib, kw, code):
    f, mag = (ctypes.c_double * 32)(), ctypes.c_double()
    sc = tv.rope_scaling(**kw)
    assert tv.load().tv_rope_frequencies(ctypes.byref(sc), 64, f, ctypes.byref(mag)) == code
    if code != tv.TV_OK:
        assert tv.load().tv_rope(ctypes.byref(rope_args(scaling=sc)), None) == code
        assert tv.load().tv_norm_rope(ctypes.byref(norm_args(scaling=sc)), None) == code


@pytest.mark.parametrize("rot", [2, 10, 64, 128, 512])
@pytest.mark.parametrize("kind,factor", [("plain", 1.0), ("linear", 4.0), ("ntk", 8.0),
                                         ("yarn", 1.0), ("yarn", 40.0), ("wavelength", 8.0)])
@pytest.mark.parametrize("base,context", [(10000.0, 4096), (500000.0, 8192)])
def test_frequencies(tvlib, rot, kind, factor, base, context):
    sc = tv.rope_scaling(base=base, kind=getattr(tv, "ROPE_" + kind.upper()), factor=factor,
                         original_context=context)
    f, mag = tv.rope_frequencies(sc, rot)
    np.testing.assert_allclose(f, dm.frequencies(rot, base, kind, factor, context), rtol=1e-13)
    assert mag == pytest.approx(dm.magnitude(kind, factor), rel=1e-15)
    if factor == 1.0:                      # nothing is stretched
        np.testing.assert_array_equal(f, tv.rope_frequencies(tv.rope_scaling(base=base), rot)[0])


def test_a_given_magnitude(tvlib):
    assert tv.rope_frequencies(tv.rope_scaling(magnitude=0.75), 8)[1] == 0.75
    assert tv.rope_frequencies(tv.rope_scaling(kind=tv.ROPE_YARN, factor=8, magnitude=2.0),
                               8)[1] == 2.0


def norm_args(**kw):
    a = tv.NormRopeArgs()
    a.B, a.T, a.H, a.d_nope, a.d_rope, a.d_latent, a.rot_dim = 2, 10, 4, 32, 16, 64, 16
    a.dt, a.eps = tv.TV_F32, 1e-6
    a.q, a.q_stride_token, a.q_stride_head = FAKE, 192, 48
    a.kv, a.kv_stride_token = FAKE + M, 80
    a.q_start, a.prefix_len = FAKE + 2 * M, FAKE + 3 * M
    a.q_nope, a.q_pe, a.c_kv, a.k_pe = (FAKE + i * M for i in range(4, 8))
    a.ckv_row_stride, a.kpe_row_stride = 64, 16
    a.cache = tv.CacheLayout(FAKE + 8 * M, 64, 8, 0, 1024)
    a.scaling = tv.rope_scaling()
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=8), BAD), (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(H=0), BAD),
    (dict(d_nope=-1), BAD), (dict(d_rope=1), BAD), (dict(d_latent=0), BAD),
    (dict(rot_dim=18), BAD), (dict(rot_dim=3), BAD), (dict(d_latent=65536), UNS),
    (dict(layout=-1), BAD), (dict(dt=7), BAD), (dict(eps=-1e-6), BAD),
    (dict(eps=float("nan")), BAD), (dict(q=None, kv=None), BAD), (dict(q_start=None), BAD),
    (dict(q_pe=None), BAD), (dict(q_nope=None), BAD), (dict(c_kv=None), BAD),
    (dict(q_stride_head=-1), BAD), (dict(kv_stride_token=1 << 31), BAD),
    (dict(ckv_row_stride=63), BAD), (dict(kpe_row_stride=15), BAD), (dict(q=FAKE + 1), BAD),
    (dict(c_kv=FAKE + 6 * M + 2), BAD), (dict(cache=tv.CacheLayout(FAKE, 64, 8, 0, 0)), BAD),
    (dict(cache=tv.CacheLayout(FAKE, 0, 8, 0, 1024)), BAD),
    (dict(cache=tv.CacheLayout(None, 64, 0, 0, 1024)), BAD),
    (dict(q_pe=FAKE), BAD), (dict(c_kv=FAKE + M), BAD), (dict(q_pe=FAKE + 4 * M + 64), BAD),
    (dict(k_pe=FAKE + 5 * M + 64), BAD), (dict(q_weight=FAKE + 5 * M), BAD),
    (dict(T=0, q_start=None), tv.TV_OK), (dict(B=0, q_start=None), tv.TV_OK),
])
def test_norm_rope_arguments(tvlib, kw, code):
    assert tv.load().tv_norm_rope(ctypes.byref(norm_args(**kw)), None) == code
    assert (code == tv.TV_OK) == (not tv.load().tv_last_error())


def shared_args(**kw):
    a = tv.SharedArgs()
    a.B, a.H, a.Q, a.d_latent, a.d_rope, a.scale = 4, 16, 3, 512, 64, 0.07
    a.dt, a.out_dt = tv.TV_BF16, tv.TV_F32
    a.q_latent, a.q_pe, a.c_kv, a.k_pe = FAKE, FAKE + M, FAKE + 16 * M, FAKE + 32 * M
    a.ckv_row_stride, a.kpe_row_stride = 512, 64
    a.cache = tv.CacheLayout(FAKE + 40 * M, 64, 32, 0, 4096)
    a.prefix_len, a.max_prefix_len, a.G = FAKE + 41 * M, 1000, 2
    a.group_start, a.shared_len, a.anc = (FAKE + i * M for i in (42, 43, 44))
    a.out, a.lse = FAKE + 45 * M, FAKE + 47 * M
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=8), BAD), (dict(B=-1), BAD), (dict(H=0), BAD), (dict(Q=0), BAD),
    (dict(Q=65), UNS), (dict(max_prefix_len=-1), BAD), (dict(G=-1), BAD), (dict(G=5), BAD),
    (dict(scale=0.0), BAD), (dict(scale=float("nan")), BAD), (dict(scale=1e31), BAD),
    (dict(dt=tv.TV_F32), UNS), (dict(out_dt=3), BAD), (dict(d_latent=256), UNS),
    (dict(d_rope=32), UNS), (dict(H=1 << 20), UNS), (dict(B=1 << 24, H=64), UNS),
    (dict(max_prefix_len=(1 << 30) + 1), UNS), (dict(q_pe=None), BAD), (dict(out=None), BAD),
    (dict(group_start=None), BAD), (dict(shared_len=None), BAD),
    (dict(cache=tv.CacheLayout(FAKE + 40 * M, 64, 32, 0, 0)), BAD),
    (dict(cache=tv.CacheLayout(FAKE + 40 * M, 64, 32, 0, (1 << 31) - 64)), BAD),
    (dict(cache=tv.CacheLayout(FAKE + 40 * M, 32, 32, 0, 4096)), UNS),
    (dict(cache=tv.CacheLayout(FAKE + 40 * M, 64, 0, 0, 4096)), BAD),
    (dict(cache=tv.CacheLayout(None, 64, 0, 0, 4096)), BAD),
    (dict(cache=tv.CacheLayout(None, 64, 0, 1025, 4096)), BAD),
    (dict(ckv_row_stride=511), BAD), (dict(ckv_row_stride=516), BAD),
    (dict(kpe_row_stride=56), BAD), (dict(c_kv=FAKE + 16 * M + 8), BAD),
    (dict(out=FAKE + 45 * M + 4), BAD), (dict(lse=FAKE + 47 * M + 2), BAD),
    (dict(out=FAKE), BAD), (dict(lse=FAKE + 45 * M + 64), BAD), (dict(lse=FAKE + 43 * M), BAD),
    (dict(out=FAKE + 41 * M), BAD), (dict(B=0, G=0, q_latent=None), tv.TV_OK),
])
def test_shared_attn_arguments(tvlib, kw, code):
    lib, a = tv.load(), shared_args(**kw)
    assert lib.tv_shared_attn(ctypes.byref(a), None, 0, None) == code
    assert (code == tv.TV_OK) == (not lib.tv_last_error())
    assert lib.tv_shared_attn_workspace_size(ctypes.byref(a)) == 0


def test_shared_attn_workspace(tvlib):
    lib, a = tv.load(), shared_args()
    n = lib.tv_shared_attn_workspace_size(ctypes.byref(a))
    assert n > 2 * 4 * 3 * 16 * 2052
    for ws, size in ((None, n), (FAKE + 128, n), (FAKE, n - 1)):
        assert lib.tv_shared_attn(ctypes.byref(a), ws, size, None) == tv.TV_ERR_WORKSPACE
    assert lib.tv_shared_attn_workspace_size(ctypes.byref(shared_args(G=0))) <= n


def test_shared_fault_hook_arguments(tvlib):
    lib = tv.load()
    assert lib.tv_testing_set_shared_fault(2, 0, None) == BAD
    assert lib.tv_testing_set_shared_fault(0, 0, None) == tv.TV_OK


def token_args(**kw):
    a = tv.TokenArgs()
    a.B, a.vocab, a.logits_dt, a.logits_row_stride = 3, 1000, tv.TV_F32, 1000
    a.logits, a.uniforms, a.tokens = FAKE, FAKE + M, FAKE + 2 * M
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=8), BAD), (dict(B=-1), BAD), (dict(vocab=0), BAD),
    (dict(vocab=(1 << 18) + 1, logits_row_stride=1 << 19), UNS), (dict(B=1 << 24), UNS),
    (dict(logits_dt=2), BAD), (dict(logits_row_stride=999), BAD),
    (dict(logits_row_stride=1 << 31), BAD), (dict(logits=None), BAD),
    (dict(logits=FAKE + 2), BAD), (dict(uniforms=None), BAD), (dict(tokens=None), BAD),
    (dict(tokens=FAKE + 4 * 2999), BAD), (dict(kept=FAKE + M + 8), BAD),
    (dict(kept=FAKE + 2 * M + 8), BAD), (dict(top_k=FAKE + 2 * M), BAD),
    (dict(min_p=FAKE + 2 * M - 8), BAD), (dict(B=0, logits=None), tv.TV_OK),
])
def test_token_sample_arguments(tvlib, kw, code):
    assert tv.load().tv_token_sample(ctypes.byref(token_args(**kw)), None) == code
    assert (code == tv.TV_OK) == (not tv.load().tv_last_error())
