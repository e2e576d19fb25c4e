"""What the tensor-core attention kernel rests on and no result shows: read from its source.  CPU only."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _source():
    with open(os.path.join(ROOT, "rmsnorm_fwd_bwd_03_gb300", "csrc", "attn8_many.cu"), encoding="utf-8") as f:
        return f.read()


def _stores_in_order(text):
    """Whether every second computation of a step's weights waits for the stores of the first."""
    step = text[text.index("const auto weigh = [&]"):]
    calls = [m.start() for m in re.finditer(r"\bweigh\(\);", step)]
    return len(calls) == 2 and "tm_wait_st();" in step[calls[0]:calls[1]]


def test_stores_to_the_same_columns_of_tensor_memory_are_ordered():
    """A row that is computed anew stores its weights twice; only tcgen05.wait::st orders a thread's stores."""
    text = _source()
    assert _stores_in_order(text)
    planted = re.sub(r"tm_wait_st\(\);[^\n]*\n(\s*weigh\(\);)", r"\1", text)
    assert planted != text and not _stores_in_order(planted)


def _constant(text, name):
    return int(re.search(rf"\b{name} = (\d+)", text)[1])


def test_no_launch_with_fewer_registers_than_the_groups_share():
    """setmaxnreg.inc waits for registers that the block was not launched with: the host refuses such a kernel."""
    text = _source()
    launch = _constant(text, "kRegsLaunch")
    assert 2 * _constant(text, "kRegsRows") + 2 * _constant(text, "kRegsConv") + _constant(text, "kRegsMma") <= 5 * launch
    assert _constant(text, "kManyThreads") * launch <= 65536
    host = text[text.index("gbln_status many_go("):]
    asks = re.search(r"cudaFuncGetAttributes\(&is, attn8_many<D, FMT>\) != cudaSuccess \|\| is\.numRegs < kRegsLaunch[^{]*\{[^}]*return GBLN_ERR_CUDA;", host)
    assert asks and asks.end() < host.index("attn8_many<D, FMT><<<")
