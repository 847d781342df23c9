"""The 4-bit cache's entry points without a GPU: sizes, refusals of bad
arguments with the documented status before any CUDA call, and the binding's
own checks. Fake pointers stand for device memory, so a call that passes the
host checks fails at the device check."""
import ctypes

import numpy as np
import pytest
import torch

import cache_ref
from exact_io_aware_attention_gb300 import binding
from exact_io_aware_attention_gb300 import build as fa_build

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA = 0, 1, 2, 3, 4
PASSED_HOST_CHECKS = (INVALID, CUDA)
A = 0x10000


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return binding.load_library()


def cache(data=A, pages=8, heads=2, page=64, d=64, dtype=binding.FA_BF16, reserved=0):
    return binding.FaCache(data, pages, heads, page, d, dtype, reserved)


def rows(H=2, N=5, d=64, dtype=binding.FA_BF16, ptr=A, sn=None):
    return binding.FaTensor(ptr, H * N * d, N * d, d if sn is None else sn, dtype, 0)


def call_rows(lib, name="fa_cache_write", c=None, k=None, v=None, table=A, stride=4, pages=4,
              start=A, counts=None, B=3, N=5):
    c = cache() if c is None else c
    d = c.d if c.d in (64, 96, 128, 256) else 64
    k = rows(N=max(N, 1), d=d) if k is None else k
    v = rows(N=max(N, 1), d=d) if v is None else v
    return getattr(lib, name)(c, k, v, table, stride, pages, start, counts, B, N, None)


def call_fwd(lib, q=None, c=None, table=A, stride=4, pages=400, lengths=A, counts=None, o=None,
             lse=A, B=3, Hq=4, Nq=5, causal=1, scale=0.1, ws=A, ws_bytes=1 << 40):
    c = cache() if c is None else c
    q = rows(H=4) if q is None else q
    o = rows(H=4) if o is None else o
    return lib.fa_cache_forward(q, c, table, stride, pages, lengths, counts, o, lse, B, Hq, Nq,
                                causal, scale, ws, ws_bytes, None)


def test_cache_bytes(lib):
    # 5 bits a channel of K and of V
    assert lib.fa_cache_bytes(10, 3, 48, 96) == 10 * 3 * 48 * 96 * 2 * 5 // 8
    assert lib.fa_cache_bytes(1, 1, 16, 256) == 16 * 320
    for bad in ((0, 1, 16, 64), (1, 0, 16, 64), (1, 1, 8, 64), (1, 1, 24, 64), (1, 1, 0, 64),
                (1, 1, 16, 80), (1, 1, 16, 0), (-1, 1, 16, 64), (1, 1, 1 << 25, 64)):
        assert lib.fa_cache_bytes(*bad) == 0


BAD_CACHES = [
    (dict(data=None), INVALID), (dict(reserved=1), INVALID), (dict(pages=0), INVALID),
    (dict(heads=0), INVALID), (dict(page=0), INVALID), (dict(page=-16), INVALID),
    (dict(page=24), UNSUPPORTED), (dict(d=80), UNSUPPORTED),
    (dict(dtype=binding.FA_F32), UNSUPPORTED), (dict(data=A + 8), MISALIGNED),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
@pytest.mark.parametrize("entry", ["fa_cache_write", "fa_cache_read", "fa_cache_forward"])
def test_bad_caches_are_refused(lib, entry, kw, status):
    if entry == "fa_cache_forward":
        assert call_fwd(lib, c=cache(**kw)) == status
    else:
        assert call_rows(lib, entry, c=cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), INVALID), (dict(start=None), INVALID), (dict(pages=0), INVALID),
    (dict(stride=-4), INVALID), (dict(B=-1), INVALID), (dict(N=-1), INVALID),
    (dict(k=rows(ptr=None)), INVALID), (dict(k=rows(dtype=binding.FA_F16)), UNSUPPORTED),
    (dict(v=rows(dtype=binding.FA_F32)), UNSUPPORTED), (dict(v=rows(ptr=A + 2)), MISALIGNED),
    (dict(k=rows(sn=60)), MISALIGNED), (dict(k=rows(sn=0)), UNSUPPORTED),
    (dict(table=A + 2), MISALIGNED), (dict(start=A + 1), MISALIGNED),
    (dict(counts=A + 2), MISALIGNED), (dict(pages=(1 << 24) // 64 + 1), UNSUPPORTED),
    (dict(B=1 << 28, N=5), UNSUPPORTED), (dict(B=1 << 30, N=1 << 30), UNSUPPORTED),
    (dict(B=0), OK), (dict(N=0), OK),
])
@pytest.mark.parametrize("entry", ["fa_cache_write", "fa_cache_read"])
def test_rows_arguments(lib, entry, kw, status):
    assert call_rows(lib, entry, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(lengths=None), INVALID), (dict(lse=None), INVALID), (dict(ws=None), INVALID),
    (dict(table=None), INVALID), (dict(q=rows(H=4, ptr=None)), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=-1.0), INVALID),
    (dict(Hq=3), INVALID), (dict(B=-1), INVALID), (dict(Nq=-1), INVALID),
    (dict(q=rows(H=4, dtype=binding.FA_F16)), UNSUPPORTED),
    (dict(o=rows(H=4, dtype=binding.FA_F16)), UNSUPPORTED),
    (dict(q=rows(H=4, sn=0)), UNSUPPORTED), (dict(o=rows(H=4, sn=68)), MISALIGNED),
    (dict(lse=A + 4), MISALIGNED), (dict(ws=A + 128), MISALIGNED),
    (dict(lengths=A + 2), MISALIGNED), (dict(counts=A + 1), MISALIGNED),
    (dict(pages=(1 << 24) // 64 + 1), UNSUPPORTED), (dict(B=1 << 28), UNSUPPORTED),
    (dict(B=1 << 30, Hq=1 << 30, Nq=1 << 30), UNSUPPORTED),
    (dict(B=0), OK), (dict(Nq=0), OK), (dict(Hq=0), OK),
])
def test_forward_arguments(lib, kw, status):
    assert call_fwd(lib, **kw) == status


def test_good_arguments_reach_the_device_check(lib):
    assert call_rows(lib) in PASSED_HOST_CHECKS
    assert call_rows(lib, "fa_cache_read", counts=A) in PASSED_HOST_CHECKS
    assert call_rows(lib, B=1, stride=-7) in PASSED_HOST_CHECKS  # the stride of one row is unused
    assert call_fwd(lib) in PASSED_HOST_CHECKS
    assert call_fwd(lib, o=rows(H=4, dtype=binding.FA_F32)) in PASSED_HOST_CHECKS


def test_refusals_are_explained(lib):
    call_fwd(lib, Hq=3)
    assert b"query heads" in lib.fa_last_error()
    call_rows(lib, c=cache(page=24))
    assert b"page size" in lib.fa_last_error()
    assert lib.fa_status_string(6) == b"FA_ERR_BAD_INDEX"


def test_workspace_bytes_of_invalid_sizes(lib):
    for bad in ((-1, 1, 1, 64, 4096), (4, 0, 1, 64, 4096), (4, 2, -1, 64, 4096),
                (4, 2, 1, 65, 4096), (4, 2, 1, 64, -1), (4, 2, 1, 64, 16)):
        assert lib.fa_cache_forward_workspace_bytes(*bad) == 0


def test_binding_refuses_what_no_cache_holds():
    with pytest.raises(ValueError, match="bf16 or fp16"):
        binding.KVCache4(4, 2, 64, dtype=torch.float32)
    for bad in (dict(d=80), dict(page_size=20), dict(num_pages=0), dict(heads=-1)):
        with pytest.raises(ValueError, match="no cache"):
            binding.KVCache4(**{**dict(num_pages=4, heads=2, d=64), **bad})
    with pytest.raises(ValueError, match="CUDA"):
        binding.KVCache4(4, 2, 64, device="cpu")


# -- the plain implementation the GPU tests compare with ------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_reference_quantiser_is_within_half_a_step(dtype):
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(200, 128, generator=g) * 3 + 1).to(dtype)
    u, s, lo = cache_ref.quantise(x)
    assert u.min() == 0 and u.max() == 15
    err = np.abs(cache_ref.stands_for(x) - x.double().numpy()).reshape(200, 4, 32)
    # half a step, and the rounding of s (half its last bit) at 15 steps
    eps = torch.finfo(dtype).eps
    assert (err <= s[..., None] * (0.5 + 15 * eps / 2)).all()


def test_reference_quantiser_special_groups():
    x = torch.zeros(4, 64)
    x[0] = 2.5                       # constant: s = 0
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    x[3, :32] = torch.arange(32) * 0.5
    x = x.to(torch.bfloat16)
    y = cache_ref.stands_for(x)
    assert (y[0] == 2.5).all()
    assert np.isnan(y[1, :32]).all() and (y[1, 32:] == 0).all()
    assert np.isnan(y[2, :32]).all() and (y[2, 32:] == 0).all()
    assert y[3, 0] == 0 and abs(y[3, 31] - 15.5) < 0.1
    huge = torch.full((1, 32), 3e38)
    huge[0, 0] = -3e38
    assert np.isnan(cache_ref.stands_for(huge.to(torch.bfloat16))).all()


def test_reference_attention_is_softmax():
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(2, 7, 64, generator=g).to(torch.float16) for _ in range(3))
    o, lse, _, _ = cache_ref.attend(q, k, v, 7, True, 0.125, 0.0)
    kd, vd = torch.from_numpy(cache_ref.stands_for(k)), torch.from_numpy(cache_ref.stands_for(v))
    z = 0.125 * q.double() @ kd.transpose(1, 2)
    z = z.masked_fill(torch.ones(7, 7).triu(1).bool(), float("-inf"))
    assert np.allclose(o, (torch.softmax(z, -1) @ vd).numpy(), atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(z, -1).numpy(), atol=1e-12)
