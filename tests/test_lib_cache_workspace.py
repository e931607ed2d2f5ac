"""The workspace of the prompt and cache calls has to lie on the tensors' device (CPU:
tensors that say they are on a CUDA device, and a launcher that only notes the call)."""
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa


class OnCuda0(torch.Tensor):
    """A CPU tensor that calls itself one of cuda:0."""

    index = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.index


class OnCuda1(OnCuda0):
    index = 1


def on(cls, *shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype).as_subclass(cls)


@pytest.fixture
def launched(monkeypatch):
    from block_diffusion_speculative_attn_gb300 import build
    build.build()
    names = []
    monkeypatch.setattr(bdsa, "_launch", lambda fn, name, index, *args: names.append(name))
    return names


def chunk(workspace):
    bf = torch.bfloat16
    q, cache = on(OnCuda0, 3, 2, 64, dtype=bf), on(OnCuda0, 32, 1, 64, dtype=bf)
    table, lens, cu = on(OnCuda0, 2, 2), on(OnCuda0, 2), on(OnCuda0, 3)
    bdsa.chunk_attn_paged(q, cache, cache, table, lens, cu, page_size=16, scale=1.0,
                          out=torch.zeros_like(q), workspace=workspace)


def fork(workspace):
    row, table, state = on(OnCuda0, 2), on(OnCuda0, 2, 3), on(OnCuda0, 2)
    out = {k: on(OnCuda0, 2, 3) if k == "block_table" else on(OnCuda0, 2) for k in bdsa.FORK_KEYS}
    bdsa.cache_fork(row, row, table, row, on(OnCuda0, 8), state, page_size=16, out=out,
                    workspace=workspace)


@pytest.mark.parametrize("call", [chunk, fork])
def test_workspace_on_another_device_is_refused(call, launched):
    u8 = torch.uint8
    for bad in (on(OnCuda1, 1 << 12, dtype=u8), torch.zeros(1 << 12, dtype=u8),
                on(OnCuda0, 64, 64, dtype=u8).t()):
        with pytest.raises(ValueError, match="workspace"):
            call(bad)
    assert launched == []
    call(on(OnCuda0, 1 << 12, dtype=u8))
    assert len(launched) == 1
