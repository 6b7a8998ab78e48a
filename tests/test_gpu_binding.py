"""The binding of the calls for candidate continuations on the GPU: workspaces that callers bring."""
import pytest
import torch

from test_gpu_candidates import Tree, check, pkv  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_a_workspace_of_any_shape_counts_by_its_bytes(pkv):  # noqa: F811
    b = Tree(40, [70, 900], [5, 3], 8, 2)
    want, tol = b.expected()
    check(b.run(pkv, workspace=torch.empty(64, 1 << 20, dtype=torch.uint8, device="cuda")), want, tol)
    check(b.run(pkv, workspace=torch.empty(1 << 26, 1, dtype=torch.uint8, device="cuda")), want, tol)
    for small in ((16, 16), (4, 0), (0,)):
        with pytest.raises(pkv.PkvError) as e:
            b.run(pkv, workspace=torch.empty(small, dtype=torch.uint8, device="cuda"))
        assert e.value.status in (pkv.PKV_ERR_NO_MEMORY, pkv.PKV_ERR_INVALID_ARG)
    with pytest.raises(ValueError, match="workspace"):
        b.run(pkv, workspace=torch.zeros((), dtype=torch.uint8, device="cuda"))
