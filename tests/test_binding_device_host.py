"""The pruned-layer calls make their tensors' device current before the library is entered (CPU only: the library and the
device switch are stand-ins, the tensors hold no memory)."""
import contextlib
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import activation_sparsification_amd._binding as B

CALLS = {
    "prepare_weight": lambda x, pw, cfg: B.prepare_weight(x),
    "prune_nm": lambda x, pw, cfg: B.prune_nm(x, cfg),
    "prune_nm by name": lambda x, pw, cfg: B.prune_nm(cfg=cfg, x=x),
    "sparse_ffn_relu2_prefill": lambda x, pw, cfg: B.sparse_ffn_relu2_prefill(x, x, x),
    "EtaCalibration.add": lambda x, pw, cfg: B.EtaCalibration(8, x.device).add(x, x[:, 0].int()),
    "EtaCalibration.table": lambda x, pw, cfg: B.EtaCalibration(8, x.device).table(),
    "eta_lookup": lambda x, pw, cfg: B.eta_lookup(x[0].float(), x[:, 0].int()),
    "prepare_amber": lambda x, pw, cfg: B.prepare_amber(x),
    "encode_meta": lambda x, pw, cfg: B.encode_meta(x.to(torch.uint8), 2, 4),
    "decode_meta": lambda x, pw, cfg: B.decode_meta(x.int(), 64, 2, 4),
    "sparse_linear_decode": lambda x, pw, cfg: B.sparse_linear_decode(x, pw, cfg),
    "sparse_linear_decode_static": lambda x, pw, cfg: B.sparse_linear_decode_static(x, pw, cfg),
    "sparse_linear_prefill": lambda x, pw, cfg: B.sparse_linear_prefill(x, pw, cfg),
    "prepare_weight_fp8": lambda x, pw, cfg: B.prepare_weight_fp8(x),
    "sparse_linear_prefill_fp8": lambda x, pw, cfg: B.sparse_linear_prefill_fp8(x, pw, B.Fp8Weight(x, x[0]), cfg),
    "PreparedCall": lambda x, pw, cfg: B.PreparedCall("sparse_linear_decode", x, pw, cfg, x, None)(),
}
ASKS = ("workspace_bytes", "meta_row_bytes")        # sizes, asked of the host


class Library:
    """Stands for libspa.so: every entry returns 0 and notes which device was current."""

    def __init__(self):
        self.current, self.entered = 0, []

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith(ASKS):
                return 64
            self.entered.append((name, self.current))
            return 0
        return entry

    @contextlib.contextmanager
    def switch(self, device):
        was, self.current = self.current, device.index
        yield
        self.current = was


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("index", [0, 1])
def test_launches_go_to_the_tensors_device(monkeypatch, name, index):
    library = Library()
    monkeypatch.setattr(B, "lib", lambda: library)
    monkeypatch.setattr(B, "_ptr", lambda t: None)
    monkeypatch.setattr(B, "_stream", lambda device: ctypes.c_void_p(0))
    monkeypatch.setattr(B, "_dev", lambda t: t.device)
    monkeypatch.setattr(B, "_WS_CACHE", {})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: library.current)
    monkeypatch.setattr(torch.cuda, "device", library.switch)
    with FakeTensorMode(allow_non_fake_inputs=True):
        x = torch.empty((4, 64), dtype=torch.bfloat16, device=f"cuda:{index}")
        pw = B.PreparedWeight(x, None, None, None)
        CALLS[name](x, pw, B.PruneConfig(2, 4))
    assert library.entered and all(device == index for _, device in library.entered), library.entered
    assert library.current == 0
