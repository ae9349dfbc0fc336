"""The layer operators' binding on tensors that it has to refuse, without a GPU: host tensors,
and no call gets as far as a launch."""
import pytest
import torch

import bit_floating_point_amd as F
from bit_floating_point_amd import _lib as L
from bit_floating_point_amd import layer as Y

E4M3 = F.grid_minifloat(4, 3)


@pytest.fixture(autouse=True)
def _no_stream(monkeypatch):
    monkeypatch.setattr(Y, "_stream", lambda dev: None)


def views(dtype):
    """[n, k] and [batch, n, k] tensors whose rows, or matrices, share memory."""
    row = torch.zeros(1, 256, dtype=dtype)
    return {"expanded rows": row.expand(64, 256), "overlapping rows": torch.zeros(8192, dtype=dtype).as_strided((32, 256), (128, 1)),
            "unfolded": torch.zeros(1024, dtype=dtype).unfold(0, 256, 8), "expanded rows of matrices": row.expand(3, 64, 256)}


@pytest.mark.parametrize("name", list(views(torch.float32)))
def test_quantize_block_of_overlapping_rows(name):
    """A row stride below k: the kernel would read past the end."""
    with pytest.raises(F.FP4Error) as e:
        F.fp4_quantize_block(views(torch.float32)[name], E4M3)
    assert e.value.status == L.FP4_ERR_INVALID_ARG


@pytest.mark.parametrize("name", list(views(torch.uint8)))
def test_quantize_block_into_overlapping_rows(name):
    packed = views(torch.uint8)[name]
    with pytest.raises(F.FP4Error) as e:
        F.fp4_quantize_block(torch.zeros(packed.shape), E4M3, packed=packed)
    assert e.value.status == L.FP4_ERR_INVALID_ARG


@pytest.mark.parametrize("stride", [(0, 256, 1), (256, 256, 1), (63 * 256, 256, 1), (512, 1024, 1)])
def test_quantize_block_into_overlapping_matrices(stride):
    packed = torch.zeros(3 * 64 * 768, dtype=torch.uint8).as_strided((3, 64, 256), stride)
    with pytest.raises(F.FP4Error) as e:
        F.fp4_quantize_block(torch.zeros(3, 64, 256), E4M3, packed=packed)
    assert e.value.status == L.FP4_ERR_INVALID_ARG


@pytest.mark.parametrize("w_stride,p_stride", [((64 * 256, 256, 1), (256, 768, 1)), ((0, 256, 1), (64 * 256, 256, 1)),
                                               ((256, 768, 1), (64 * 320, 320, 1)), ((64 * 256, 256, 1), (512, 768, 1))])
def test_quantize_block_takes_other_layouts(monkeypatch, w_stride, p_stride):
    """Interleaved matrices, padded rows, and one matrix read three times reach the library as they
    are."""
    given = []
    monkeypatch.setattr(Y, "_call", lambda name: lambda *a: given.append(a) or 0)
    w = torch.zeros(3 * 64 * 768).as_strided((3, 64, 256), w_stride)
    packed = torch.zeros(3 * 64 * 768, dtype=torch.uint8).as_strided((3, 64, 256), p_stride)
    F.fp4_quantize_block(w, E4M3, packed=packed)
    _, _, batch, n, k, ldw, stride_w, _, _, ldp, stride_p, _, _ = given[0]
    assert (batch, n, k, ldw, stride_w, ldp, stride_p) == (3, 64, 256, w_stride[1], w_stride[0], p_stride[1], p_stride[0])


def test_quantize_block_of_one_row(monkeypatch):
    """The stride of a single row means nothing."""
    given = []
    monkeypatch.setattr(Y, "_call", lambda name: lambda *a: given.append(a) or 0)
    F.fp4_quantize_block(torch.zeros(256).as_strided((1, 256), (0, 1)), E4M3)
    F.fp4_quantize_block(torch.zeros(512).as_strided((2, 1, 256), (256, 8, 1)), E4M3)
    assert given[0][5] == 256 and given[1][5] == 256


# the library's own rule (device pointers are never dereferenced before it)
@pytest.mark.parametrize("batch,ldp,stride_p,status", [
    (2, 256, 0, L.FP4_ERR_INVALID_ARG), (2, 256, 63 * 256, L.FP4_ERR_INVALID_ARG), (3, 512, 256, L.FP4_ERR_INVALID_ARG),
    (3, 768, 128, L.FP4_ERR_INVALID_ARG), (65, 512, 520, L.FP4_ERR_INVALID_ARG), (1 << 20, 256, 8, L.FP4_ERR_INVALID_ARG),
    (1, 256, 0, L.FP4_ERR_ALIGNMENT), (2, 256, 63 * 256 + 256, L.FP4_ERR_ALIGNMENT), (3, 768, 256, L.FP4_ERR_ALIGNMENT),
    (3, 768, 512, L.FP4_ERR_ALIGNMENT), (1 << 20, 256 << 20, 256, L.FP4_ERR_ALIGNMENT), (1 << 20, 256, 64 * 256, L.FP4_ERR_ALIGNMENT)])
def test_overlap_rule(batch, ldp, stride_p, status):
    """Codes of different matrices may not share memory.  Layouts that pass stop at the scales'
    alignment, so no case launches anything."""
    got = Y._call("fp4_quantize_block")(0x10000, L.FP4_F32, batch, 64, 256, 256, 64 * 256, E4M3, 0x10000, ldp, stride_p, 0x10002, None)
    assert got == status
    assert (b"overlap" in L.lib().fp4_last_error()) == (status == L.FP4_ERR_INVALID_ARG)


# fp4_route counts in the caller's workspace: it has to be memory of the logits' device, as large
# as it says.
@pytest.mark.parametrize("workspace", [torch.empty(1 << 20, dtype=torch.uint8, device="meta"),
                                       torch.zeros(1, dtype=torch.uint8).expand(1 << 20),
                                       torch.zeros(8192, dtype=torch.int32).as_strided((1 << 10, 64), (4, 1)),
                                       torch.zeros(1 << 20, dtype=torch.uint8)[::2]])
def test_route_workspace(workspace):
    with pytest.raises(ValueError, match="workspace"):
        F.fp4_route(torch.zeros(4096, 64), 8, workspace=workspace)


def test_route_takes_a_workspace(monkeypatch):
    """A workspace that is large enough is used, a small one replaced, none needed for few tokens."""
    size, given = Y._call("fp4_route_workspace_size"), []
    monkeypatch.setattr(Y, "_call", lambda name: size if name.endswith("size") else lambda *a: given.append(a) or 0)
    workspace = torch.zeros(1 << 20, dtype=torch.uint8)
    F.fp4_route(torch.zeros(4096, 64), 8, workspace=workspace)
    F.fp4_route(torch.zeros(4096, 64), 8, workspace=workspace[:64])
    F.fp4_route(torch.zeros(4, 64), 8, workspace=workspace)
    assert given[0][1] == workspace.data_ptr() and given[0][2] == size(4096, 64, 8)
    assert given[1][1] != workspace.data_ptr() and given[2][1] is None
