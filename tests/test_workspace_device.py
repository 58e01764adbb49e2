"""The MXFP4 helpers keep workspace sizes by the device the library answers for, the current one, also where the tensors are
on another: a product's plan, and with it its workspace, follows the current device's compute units.  Without a GPU: a
library and a tensor that stand in for them."""

import fp8_blockwise_quantized_amd.mx as mx


class Lib:
    sizes = {0: 1024, 1: 4096}
    current = 0

    def fp8bq_gemm_mxfp4_workspace_size(self, M, N, K):
        return self.sizes[self.current]


class Tensor:
    is_cuda = True

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device

    def new_empty(self, n, dtype):
        return n


def test_sizes_follow_the_current_device(monkeypatch):
    lib = Lib()
    monkeypatch.setattr(mx, "lib", lambda: lib)
    monkeypatch.setattr(mx, "_current_device", lambda: lib.current, raising=False)
    mx._ws_bytes.cache_clear()
    try:
        for lib.current in (0, 1, 0, 1):
            for device in (0, 1):
                assert mx._space("fp8bq_gemm_mxfp4_workspace_size", Tensor(device), 64, 2048, 11264) == Lib.sizes[lib.current]
    finally:
        mx._ws_bytes.cache_clear()
