"""What a call on a stream of the caller's allocates belongs to that stream."""

import pytest
import torch

pytestmark = pytest.mark.gpu

B, H, L, D = 1, 2, 128, 64


@pytest.fixture(scope="module")
def lz():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_linear_sliding_chunkwise_b200 import lizard
    return lizard


def _calls(lz):
    """Each entry point that allocates, as a call that takes a stream and gives its tensors."""
    gen = torch.Generator().manual_seed(0)

    def normal(*shape):
        return torch.randn(*shape, generator=gen).cuda()

    q, k, v, g, dout = (normal(B, H, L, D) for _ in range(5))
    wq, wk, alpha = normal(H, D, D // 2), normal(H, D, D // 2), normal(H)
    kw = dict(window=32, fmap_wq=wq, fmap_wk=wk, alpha=alpha)
    q1, k1, v1, g1 = (normal(B, H, D) for _ in range(4))
    one = [normal(B, H, D, D), normal(B, H, 32, D), normal(B, H, 32, D),
           torch.full((B,), 40, dtype=torch.int32, device="cuda")]      # state, caches, position: updated in place
    caches = iter([[x.clone() for x in one] for _ in range(2)])
    seg, dec = normal(2, B, H, D, D), -normal(2, B, H, D).abs()

    def tensors(r):
        return [t for t in (r.values() if isinstance(r, dict) else r) if t is not None]

    return dict(
        attn_fwd=lambda **s: tensors(lz.attn_fwd(q, k, v, g, want_lse=True, want_state=True, **kw, **s)),
        attn_bwd=lambda **s: tensors(lz.attn_bwd(q, k, v, g, dout, **kw, **s)),
        stage1_step=lambda **s: tensors(lz.stage1_step(q, k, v, g, dout, want_o=True, **kw, **s)),
        decode_step=lambda **s: [lz.decode_step(q1, k1, v1, g1, *next(caches), fmap_wq=wq, fmap_wk=wk, alpha=alpha,
                                                **s)],
        segment_state=lambda **s: list(lz.segment_state(k, v, g, window=32, fmap_wk=wk, **s)),
        chain_states=lambda **s: [lz.chain_states(seg, dec, 1, **s)])


def _spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.nbytes) for t in tensors]


def _overlap(x, y):
    return [(a, b) for a in x for b in y if a[0] < b[1] and b[0] < a[1]]


@pytest.mark.parametrize("name", ["attn_fwd", "attn_bwd", "stage1_step", "decode_step", "segment_state", "chain_states"])
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_outputs_and_workspaces_belong_to_the_stream_of_the_call(lz, name, handle):
    call = _calls(lz)[name]
    s, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    plain = call()                             # `call` keeps the inputs
    sizes = [t.nbytes for t in plain]
    torch.cuda.synchronize()

    def blocks():                              # the sizes that the call wants, from the current stream's memory
        return [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]

    freed = _spans(blocks())                   # recycled at once
    out = call(stream=s.cuda_stream if handle else s)
    assert torch.cuda.current_stream() == here
    assert not _overlap(freed, _spans(out))
    s.synchronize()
    if name not in ("attn_bwd", "stage1_step"):    # (those sum over tokens with atomics)
        for x, y in zip(plain, out):
            if x.dtype == torch.float32:
                assert torch.equal(x, y)
    gone = _spans(out)
    del out
    assert not _overlap(gone, _spans(blocks()))
    torch.cuda.synchronize()


def test_the_default_stream_as_a_handle(lz):
    call = _calls(lz)["chain_states"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = call(stream=0)[0]
        assert torch.cuda.current_stream() == s
    torch.cuda.synchronize()
    assert torch.equal(out, call()[0])
