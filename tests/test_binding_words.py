"""The binding's error words on the CPU, with the CUDA queries stood in for."""
import torch

import dropless_grouped_gemm_gb300 as M


def _cpu(monkeypatch):
    monkeypatch.setattr(M, "_current_stream", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(M, "_ERR_WORDS", {})
    return torch.device("cpu")


def test_words_made_in_inference_mode_are_ordinary_tensors(monkeypatch):
    dev = _cpu(monkeypatch)
    with torch.inference_mode():
        first = M._err_word(None, dev)
        first.zero_()
    later = M._err_word(None, dev)
    assert not first.is_inference() and not later.is_inference()
    later.zero_()                       # an inference tensor would refuse this here
    assert later.data_ptr() != first.data_ptr()


def test_words_are_zero_and_handed_out_once(monkeypatch):
    dev = _cpu(monkeypatch)
    words = [M._err_word(None, dev) for _ in range(130)]
    assert len({w.data_ptr() for w in words}) == 130
    assert all(w.dtype == torch.int32 and w.tolist() == [0] for w in words)
