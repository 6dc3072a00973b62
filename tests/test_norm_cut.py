"""How a group norm is cut for a device: by its number of compute units."""
import pytest
import torch

from irregular_gather_cnn_amd import _lib as L

LAYOUTS = ["channels_first", "channels_last"]
WHOLE, JOINT, TWICE = range(3)


def desc(n, c, s, g, layout, dtype="bf16", act="none"):
    return L.deft_norm_desc(n, c, s, g, L.LAYOUTS[layout], L.ACTIVATIONS[act],
                            L.DEFT_BF16 if dtype == "bf16" else L.DEFT_F32, 1e-5)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("cus", [32, 64, 256])
def test_workgroups_that_share_a_group_fit_the_device(cus, layout, back):
    """Those that wait for each other are no more than a device of 32 (a partition of the chip) or of 256
    units holds: 1024 threads a unit forward, 512 backward."""
    most = 0
    for n in (1, 3):
        for per, g in ((1, 4), (3, 12), (32, 2), (500, 1), (2048, 1)):
            for s in (500, 3000, 20000, 150000, 1000000, 9000000):
                d = desc(n, per * g, s, g, layout)
                cut = L.deft_debug_norm_cut(d, back, cus)
                assert cut["cus"] == cus
                if cut["form"] == JOINT:
                    assert cut["slices"] * cut["threads"] <= cus * (512 if back else 1024), (n, per, g, s)
                    most = max(most, cut["slices"])
    assert most > 4  # some are that large


def test_without_a_size_the_cut_is_the_devices():
    d = desc(2, 64, 5000, 2, "channels_first")
    assert L.deft_debug_norm_cut(d, False)["cus"] >= 1
    assert {**L.deft_debug_norm_cut(d, True, 256), "cus": 0} != {**L.deft_debug_norm_cut(d, True, 32), "cus": 0}


@pytest.mark.gpu
def test_the_device_is_asked_for_its_units():
    units = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    assert L.deft_debug_norm_cut(desc(2, 64, 5000, 2, "channels_first"), False)["cus"] == units


def test_refusals():
    for d, code in ((desc(2, 64, 500, 3, "channels_first"), -2), (desc(0, 64, 500, 2, "channels_last"), -1),
                    (desc(2, 64, 0, 2, "channels_last"), -1), (desc(1, 5000, 10, 1, "channels_last"), -10)):
        with pytest.raises(L.DeftError) as e:
            L.deft_debug_norm_cut(d, False)
        assert e.value.code == code
    with pytest.raises(L.DeftError):
        L.deft_debug_norm_cut(desc(2, 64, 500, 2, "channels_first"), False, -1)


@pytest.mark.parametrize("layout,dtype,n,c,s,g,form", [
    # one workgroup a unit: all 256 at once, or a second round
    ("channels_first", "f32", 10, 96, 10688, 24, WHOLE), ("channels_first", "f32", 3, 412, 9992, 103, JOINT),
    ("channels_first", "f32", 32, 512, 2500, 32, JOINT), ("channels_last", "bf16", 40, 132, 3138, 6, WHOLE),
    ("channels_last", "bf16", 8, 640, 7000, 40, TWICE), ("channels_last", "f32", 12, 210, 1725, 35, WHOLE),
    # bf16 channels first: rounds that are 4/5 full
    ("channels_first", "bf16", 10, 335, 16678, 67, WHOLE), ("channels_first", "bf16", 4, 308, 31434, 77, JOINT),
    ("channels_first", "bf16", 34, 221, 4345, 17, JOINT)])
def test_forward_groups_that_fill_a_unit_run_in_full_rounds(layout, dtype, n, c, s, g, form):
    assert L.deft_debug_norm_cut(desc(n, c, s, g, layout, dtype), False, 256)["form"] == form
