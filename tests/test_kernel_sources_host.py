"""What the kernels' sources have to keep to and no run can show."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir, "lora_serving_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


def test_a_plan_reads_what_it_writes_by_ordinary_loads():
    """The read-only path (ld.global.nc) is undefined for memory that the kernel itself writes: counters in place, the stack of
    free pages, the block table.  So it names inputs that no plan writes, and nothing through a pointer of another name."""
    assert {re.match(r"a\.(\w+)", arg).group(1) if arg.startswith("a.") else arg
            for arg in re.findall(r"__ldg\(\s*([^()+]+?)\s*[+)]", _code("kv4_plan.cu"))} <= {"lens", "depths"}


def test_a_cluster_barrier_gathers_its_warps():
    """barrier.cluster's aligned forms are undefined unless all lanes of a warp execute them together."""
    code = _code("cluster.cuh")
    for name in ("arrive", "wait"):
        body = re.search(r"void cluster_%s\(\)\s*\{(.*?)\n?\}" % name, code, re.S).group(1)
        assert ".aligned" not in body or re.match(r"\s*__syncwarp\(\);", body)
    everywhere = {f: _code(f).count("barrier.cluster") for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))}
    assert {f for f, n in everywhere.items() if n} == {"cluster.cuh"}
