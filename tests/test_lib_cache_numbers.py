"""Numbers of the prompt and cache calls that need more than 32 bits are refused: the
C interface takes int32, and ctypes would pass on their lower bits (CPU, as in
test_lib_cache_workspace)."""
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa
from test_lib_cache_workspace import OnCuda0, launched, on  # noqa: F401

WIDE = (2 ** 32 + 16, -2 ** 32 + 16, 2 ** 31)


def chunk(**kw):
    bf = torch.bfloat16
    q, cache = on(OnCuda0, 3, 2, 64, dtype=bf), on(OnCuda0, 32, 1, 64, dtype=bf)
    a = dict(page_size=16, scale=1.0, mask_block=1, num_pages=2, sms=0)
    a.update(kw)
    bdsa.chunk_attn_paged(q, cache, cache, on(OnCuda0, 2, 2), on(OnCuda0, 2), on(OnCuda0, 3),
                          out=torch.zeros_like(q), workspace=on(OnCuda0, 64), **a)


def fork(page_size=16):
    row, out = on(OnCuda0, 2), {k: on(OnCuda0, 2) for k in bdsa.FORK_KEYS}
    out["block_table"] = on(OnCuda0, 2, 3)
    bdsa.cache_fork(row, row, on(OnCuda0, 2, 3), row, on(OnCuda0, 8), on(OnCuda0, 2),
                    page_size=page_size, out=out, workspace=on(OnCuda0, 64))


def copy(page_size=16):
    e = on(OnCuda0, 2)
    bdsa.cache_copy([on(OnCuda0, 32, 8)], e, e, e, page_size=page_size)


def compact(page_size=16):
    bdsa.cache_compact([on(OnCuda0, 32, 8)], on(OnCuda0, 2, 2), on(OnCuda0, 2),
                       on(OnCuda0, 2, 4), page_size=page_size)


@pytest.mark.parametrize("call,name", [(chunk, "page_size"), (chunk, "mask_block"),
                                       (chunk, "num_pages"), (chunk, "sms"), (fork, "page_size"),
                                       (copy, "page_size"), (compact, "page_size")])
@pytest.mark.parametrize("x", WIDE)
def test_numbers_past_32_bits(call, name, x, launched):  # noqa: F811
    with pytest.raises(ValueError):
        call(**{name: x})
    assert launched == []


@pytest.mark.parametrize("call", [chunk, fork, copy, compact])
def test_the_same_calls_go_through(call, launched):  # noqa: F811
    call()
    assert len(launched) == 1


def test_rows_past_32_bits(launched):  # noqa: F811
    """A slot of 4 GiB and 16 bytes (meta tensors: no memory)."""
    row = torch.empty((1, 1, 2 ** 32 + 16), dtype=torch.uint8, device="meta").as_subclass(OnCuda0)
    with pytest.raises(ValueError):
        bdsa.cache_write(row, row, on(OnCuda0, 1), row, row)
    assert launched == []
