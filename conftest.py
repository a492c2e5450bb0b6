"""pytest's configuration of the whole tree.

tests/test_wait_states.py counts, in every built kernel, the wait states between a matrix instruction and the use of its
result, by a table of the instructions (four per pass and four more). The MXFP4 projections add two: the scaled forms, here
on 4-bit operands, of half the passes of the 8-bit ones."""

SCALED_FP4 = {"v_mfma_scale_f32_16x16x128_f8f6f4": 8, "v_mfma_scale_f32_32x32x64_f8f6f4": 12}


def pytest_collection_modifyitems(items):
    for module in {item.module for item in items if hasattr(item, "module")}:
        if hasattr(module, "MFMA_WAIT"):
            for op, waits in SCALED_FP4.items():
                module.MFMA_WAIT.setdefault(op, waits)
