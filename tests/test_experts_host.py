"""Checks of the compiled binding that need GPU tensors but no GPU: they are made on tensors that
only say where they are."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


@pytest.fixture(scope="module")
def ex():
    from multistage_smem_pipeline_gb300 import build
    build.build()
    from multistage_smem_pipeline_gb300 import experts
    return experts


def fake(*sizes, dtype, device="cuda:0"):
    with FakeTensorMode():
        return torch.empty(*sizes, dtype=dtype, device=device)


def stored(rows=4, device="cuda:0"):
    """Codes and scales of a rows x 64 nvfp4 matrix, with scales enough for any routing of them."""
    return (fake(rows, 32, dtype=torch.uint8, device=device),
            fake(1 << 16, dtype=torch.uint8, device=device))


def test_numbers_are_not_cut_to_32_bits(ex):
    codes, scales = stored()
    assert ex.Fp4Matrix(codes, scales, cols=64, exponent=-7).exponent == -7
    for exponent in (2**32, 2**32 - 3, -2**32, 2**40 + 5, 2**63 - 1):
        with pytest.raises(ValueError, match="exponent"):
            ex.Fp4Matrix(codes, scales, cols=64, exponent=exponent)
    for cols in (2**23 + 1, 2**62, 2**63 - 1):
        with pytest.raises(ValueError, match="columns"):
            ex.Fp4Matrix(codes, scales, cols=cols)
    with pytest.raises(ValueError, match="exponent"):
        ex.fp4_quantize(fake(4, 64, dtype=torch.float16), exponent=2**32)


def routing(ex, device, experts=3, tokens=2, top_k=2):
    def ints(*sizes):
        return fake(*sizes, dtype=torch.int32, device=device)
    return ex.Routing(ints(experts + 1), ints(tokens, top_k), ints(tokens, top_k))


def test_a_routing_of_another_device_is_refused(ex):
    """A kernel would read the other GPU's offsets."""
    codes, scales = stored()
    assert ex.Fp4Matrix(codes, scales, cols=64, routing=routing(ex, "cuda:0")).groups == 3
    with pytest.raises(ValueError, match="different devices"):
        ex.Fp4Matrix(codes, scales, cols=64, routing=routing(ex, "cuda:1"))
    with pytest.raises(ValueError, match="different devices"):
        ex.fp4_quantize(fake(2, 64, dtype=torch.float16), routing=routing(ex, "cuda:1"))
    with pytest.raises(ValueError, match="one device"):
        ex.Fp4Matrix(codes, stored(device="cuda:1")[1], cols=64)


def test_the_error_word_is_the_stream_s_device_s(ex):
    """The word of the stream's own device is read, not the current one's."""
    class Stream:
        cuda_stream = 0
        asked = 0

        @property
        def device(self):
            Stream.asked += 1
            return torch.device("cuda", 63)      # there is none such

    with pytest.raises(RuntimeError):
        ex.fp4_get_device_error(Stream())
    assert Stream.asked


@pytest.mark.gpu
def test_other_threads_run_while_the_stream_is_waited_for(ex):
    import threading
    import time
    s = torch.cuda.Stream()
    assert ex.fp4_get_device_error(s) == (0, 0)
    with torch.cuda.stream(s):
        torch.cuda._sleep(600_000_000)           # 0.3 s or so
    waiter = threading.Thread(target=ex.fp4_get_device_error, args=(s,))
    waiter.start()
    steps = 0
    while waiter.is_alive():
        time.sleep(0.005)
        steps += 1
    assert steps > 10
