"""The Python binding called from several threads, without a device."""
import sys

from quantized_int8_gemm_q4_b200 import dllm


def test_the_first_call_may_come_from_two_threads(monkeypatch):
    """The stream is asked for with its helpers set up at the first call: a call that arrives between any
    two steps of that set-up finds none of them or all."""
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 40 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    monkeypatch.setattr(dllm, "_current_stream", None)
    seen = []

    def step(frame, event, arg):
        frame.f_trace_opcodes = True
        if event == "opcode" and frame.f_code is dllm._stream.__code__:
            before = dllm._current_stream
            seen.append(dllm._stream(None))  # the other thread's call, here
            dllm._current_stream = before
        return step

    old = sys.gettrace()
    sys._getframe().f_trace_opcodes = True  # opcode events are switched on with the trace function
    sys.settrace(step)
    try:
        seen.append(dllm._stream(None))
    finally:
        sys.settrace(old)
    assert len(seen) > 10 and set(seen) == {42}
