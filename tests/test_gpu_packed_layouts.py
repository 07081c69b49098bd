"""Parts of packed tensors whose extents interleave, in every order of their dimensions: rotated in place
by one call, and read back into."""
import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_cache import make_cache, status
from test_gpu_rotary import randn

pytestmark = pytest.mark.gpu
D = 64

# Shape of a tensor with two parts of H heads, and the [B, H, L, D] views of its parts.
LAYOUTS = {
    "BLPHD": (lambda B, H, L: (B, L, 2, H, D), lambda x: [x[:, :, i].transpose(1, 2) for i in range(2)]),
    "BPHLD": (lambda B, H, L: (B, 2, H, L, D), lambda x: [x[:, i] for i in range(2)]),
    "BPLHD": (lambda B, H, L: (B, 2, L, H, D), lambda x: [x[:, i].transpose(1, 2) for i in range(2)]),
    "BHPLD": (lambda B, H, L: (B, H, 2, L, D), lambda x: [x[:, :, i] for i in range(2)]),
    "BLHPD": (lambda B, H, L: (B, L, H, 2, D), lambda x: [x[:, :, :, i].transpose(1, 2) for i in range(2)]),
    "PBHLD": (lambda B, H, L: (2, B, H, L, D), lambda x: [x[0], x[1]]),
}
SIZES = [(2, 3, 5), (1, 3, 5), (2, 1, 5), (2, 3, 1), (1, 1, 1)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


@pytest.mark.parametrize("B,H,L", SIZES)
@pytest.mark.parametrize("name", LAYOUTS)
def test_rotated_in_place_by_one_call(name, B, H, L):
    shape, parts = LAYOUTS[name]
    freqs, mscale = fa.rotary_freqs(D)
    x = randn(*shape(B, H, L), dtype=torch.bfloat16)
    q, k = parts(x)
    want = fa.rotary(q.contiguous(), k.contiguous(), None, freqs, mscale)
    st = [t.stride()[:3] for t in (q, k, q, k)]
    assert fa.fa_rotary(q.data_ptr(), k.data_ptr(), q.data_ptr(), k.data_ptr(), st, None, 0, freqs.data_ptr(), D,
                        mscale, 0, 0, B, H, H, L, D, fa.FA_BF16,
                        torch.cuda.current_stream().cuda_stream) == fa.FA_OK
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("B,H,L", SIZES)
@pytest.mark.parametrize("name", LAYOUTS)
def test_read_back_into_a_packed_tensor(name, B, H, L):
    shape, parts = LAYOUTS[name]
    kc, vc, ke, ve = make_cache(B, H, D, torch.float16, True)
    bt = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    sl = torch.full((B,), L, dtype=torch.int32, device="cuda")
    k, v = randn(B, H, L, D, dtype=torch.float16), randn(B, H, L, D, dtype=torch.float16, seed=1)
    fa.cache_append(k, v, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    want = fa.cache_read(kc, vc, bt, sl, L, k_exp=ke, v_exp=ve, dtype=torch.float16)
    out = parts(torch.empty(shape(B, H, L), device="cuda", dtype=torch.float16))
    fa.cache_read(kc, vc, bt, sl, L, k_exp=ke, v_exp=ve, out=out)
    assert status() == fa.FA_OK
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    if L > 1:  # parts that meet are still refused
        with pytest.raises(fa.FaError):
            fa.cache_read(kc, vc, bt, sl, L - 1, k_exp=ke, v_exp=ve, out=(out[0][:, :, 1:], out[0][:, :, :-1]))


def _odd_ones():
    """[B, H, L, D] views whose dimensions of size 1 have strides that no row could be read by, and one
    that starts inside a 16-byte unit."""
    n = torch.randn(3 * 5 * D + 8, device="cuda").bfloat16()
    for shape, strides in (((3, 1, 5, D), (5 * D, 1, D)), ((1, 3, 5, D), (3, 5 * D, D)),
                           ((3, 5, 1, D), (5 * D, D, 7)), ((1, 1, 1, D), (1, 2, 3)), ((3, 1, 5, D), (5 * D, 0, D)),
                           ((3, 5, 1, D), (5 * D, D, 0))):
        yield torch.as_strided(n, shape, (*strides, 1))
    yield torch.as_strided(n, (3, 5, 1, D), (5 * D, D, D, 1), 1)


@pytest.mark.parametrize("i", range(7))
def test_strides_of_single_entries_mean_nothing(i):
    x = list(_odd_ones())[i]
    plain = x.clone(memory_format=torch.contiguous_format)
    B, H, L, _ = x.shape
    freqs, mscale = fa.rotary_freqs(D)
    pos = torch.arange(7, 7 + L, dtype=torch.int32, device="cuda")
    want = fa.rotary_apply(plain, pos, freqs, mscale)
    assert torch.equal(fa.rotary_apply(x, pos, freqs, mscale), want)
    q, k = x.detach().requires_grad_(), plain.detach().requires_grad_()
    qo, ko = fa.rotary(q, k, pos, freqs, mscale)
    assert torch.equal(qo, want) and torch.equal(ko, want)
    gq, = torch.autograd.grad(qo, q, x, retain_graph=True)  # the gradient has that layout too
    gk, = torch.autograd.grad(ko, k, plain)
    assert torch.equal(gq, gk)
    if i < 6:
        fa.rotary_apply(x, pos, freqs, mscale, out=x)  # in place
        assert torch.equal(x, want)
        kc, vc, ke, ve = make_cache(B, H, D, torch.bfloat16, False)
        bt = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
        sl = torch.full((B,), L, dtype=torch.int32, device="cuda")
        fa.cache_append(x, plain, kc, vc, bt, sl)
        v2 = torch.empty_like(plain)
        x.zero_()
        fa.cache_read(kc, vc, bt, sl, L, out=(x, v2))
        assert status() == fa.FA_OK and torch.equal(x, want) and torch.equal(v2, plain)
