"""The binding of drafted steps without a GPU: tensors of a device that the launch does not go to are refused."""
import os
from types import SimpleNamespace

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Device(torch.Tensor):
    """A host tensor that says it lives on a GPU, the first one unless it was moved."""

    is_cuda = property(lambda self: True)

    def get_device(self):
        return getattr(self, "at", 0)


def dev(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Device)


@pytest.fixture
def draft(monkeypatch):
    from two_level_sparse_gb300 import build

    if not os.path.exists(os.path.join(ROOT, "two_level_sparse_gb300", "libci.so")):
        build.build()
    from two_level_sparse_gb300 import draft as mod

    calls = []

    def entry(name):
        return lambda *a: calls.append(name) or 0

    size = mod.lib.ci_attn_draft_workspace_bytes
    monkeypatch.setattr(mod, "lib", SimpleNamespace(**{n: entry(n) for n in mod.SIGNATURES if not n.endswith("bytes")},
                                                    ci_attn_draft_workspace_bytes=size))
    monkeypatch.setattr(mod, "_current_device", lambda: 0)
    monkeypatch.setattr(mod, "_on", lambda stream, like: 0)
    return SimpleNamespace(mod=mod, calls=calls)


def arguments(name, bf16=torch.bfloat16):
    """Of a call with two requests and six rows: everything that can be given."""
    pool = lambda: dev(4, 2, 64 * 128, dtype=torch.uint8)  # noqa: E731
    err = dict(dev_err=dev(1))
    return {
        "ci_draft_plan": lambda: dict(length=dev(2), count=dev(2), parent=dev(2, 3), page_table=dev(2, 4), num_pages=4,
                                      req_start=dev(3), positions=dev(6), cache_pos=dev(6), mask=dev(6, 1),
                                      token=dev(2, 3), row_token=dev(6), **err),
        "ci_attn_draft": lambda: dict(q=dev(6, 4, 64, dtype=bf16), k_pool=pool(), v_pool=pool(), page_table=dev(2, 4),
                                      req_start=dev(3), length=dev(2), max_len=256, max_rows=3, scale=1.0,
                                      out=dev(6, 4, 64, dtype=bf16), mask=dev(6, 1), lse=dev(6, 4, dtype=torch.float32),
                                      workspace=dev(1 << 10, dtype=torch.uint8), **err),
        "ci_draft_accept": lambda: dict(req_start=dev(3), length=dev(2), parent=dev(2, 3), row_token=dev(6),
                                        target=dev(6), path=dev(2, 3), accepted=dev(2), next=dev(2), new_len=dev(2),
                                        cache_pos=dev(6), **err),
        "ci_slots_move": lambda: dict(pools=[pool(), pool()], row_bytes=128, scale_bytes=0, page_table=dev(2, 4),
                                      length=dev(2), path=dev(2, 3), count=dev(2), **err),
        "ci_pages_trim": lambda: dict(page_table=dev(2, 4), ref_count=dev(4), old_len=dev(2), new_len=dev(2), **err),
    }[name]()


@pytest.mark.parametrize("name", ["ci_draft_plan", "ci_attn_draft", "ci_draft_accept", "ci_slots_move", "ci_pages_trim"])
def test_tensors_of_another_device_are_refused(draft, name):
    call = getattr(draft.mod, name)
    call(**arguments(name))
    assert draft.calls == [name]
    tensors = [k for k, v in arguments(name).items() if isinstance(v, (torch.Tensor, list))]
    assert len(tensors) >= 5
    for k in tensors:
        args = arguments(name)
        (args[k][1] if isinstance(args[k], list) else args[k]).at = 1
        with pytest.raises(ValueError, match=f"{k} must live on the current device"):
            call(**args)
    if name == "ci_slots_move":  # all of them in one tensor
        args = dict(arguments(name), pools=dev(2, 4, 2, 64 * 128, dtype=torch.uint8))
        args["pools"].at = 1
        with pytest.raises(ValueError, match="pools must"):
            call(**args)
    assert draft.calls == [name]
