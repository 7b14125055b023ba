"""The gated delta rule's tensor-core kernels in the debug build
(libretnet_debug.so), whose hooks make waits run out.

With the hook on, the walks over the first (sequence, head) and the gradient
kernel's first CTA never issue the copies of their second stage, so their
waits give up after 1 ms with MMAs of the first stage issued.  The call ends
with RETNET_ERR_TIMEOUT, the CTA lets its copies and MMAs finish and frees its
tensor memory, and the next call (hook off) gives the bits of the default
library.  Nothing faults, traps or waits without a limit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TIMEOUT = 4                     # RETNET_ERR_TIMEOUT


@pytest.fixture(scope="module")
def rn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import linear_recurrent_sequence_02_b200 as lib
    from linear_recurrent_sequence_02_b200.build import build
    build()
    build(variant="debug")
    lib.load_library()
    lib.load_library(lib.DEBUG_LIB_PATH)
    return lib


def make(B, n, Hk, H, dk, dv):
    gen = torch.Generator(device="cuda").manual_seed(n + dv)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    q, k = (torch.nn.functional.normalize(normal(B, n, Hk, dk), dim=-1) for _ in range(2))
    g, beta = -torch.rand(B, n, H, generator=gen, device="cuda") * 0.1, torch.sigmoid(normal(B, n, H))
    return [x.bfloat16() for x in (q, k, normal(B, n, H, dv), g, beta, normal(B, n, H, dv))]


# walks of whole sequences and, with few heads and many chunks, of segments
@pytest.mark.parametrize("B,n,Hk,H,dk,dv", [(2, 200, 1, 2, 128, 128), (1, 2048, 1, 1, 128, 256),
                                            (1, 1500, 1, 2, 64, 64)])
@pytest.mark.parametrize("call", ["prefill", "prefill and state", "backward"])
def test_timeout_reports_and_the_context_stays_usable(rn, B, n, Hk, H, dk, dv, call):
    x = make(B, n, Hk, H, dk, dv)

    def run():
        if call == "backward":
            return rn.retnet_delta_backward(*x, algo="tensor")
        S = torch.zeros(B, H, dk, dv, device="cuda") if "state" in call else None
        out = rn.retnet_delta_chunkwise(*x[:5], state_out=S, algo="tensor")
        return (out,) if S is None else (out, S)

    want = run()
    rn.retnet_check_device_errors()
    with rn.using_library(rn.DEBUG_LIB_PATH):
        rn.retnet_check_device_errors()                      # start from a clear word
        rn.retnet_test_set_hooks(1_000_000, True)            # 1 ms limit, skip loads
        try:
            run()
            with pytest.raises(rn.RetnetError) as e:
                rn.retnet_check_device_errors()
            assert e.value.status == TIMEOUT
        finally:
            rn.retnet_test_set_hooks(2_000_000_000, False)
        got = run()                                          # hooks off: a normal call
        rn.retnet_check_device_errors()
    again = run()                                            # the default library alongside
    rn.retnet_check_device_errors()
    for a, b, c in zip(want, got, again):
        assert torch.equal(a, b) and torch.equal(a, c)
