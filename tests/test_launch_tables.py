"""What the library keeps of a launch between calls, on the CPU: the number of clusters that run at a time
goes by the whole shape of the launch, and one that cannot be had is asked again; kernels are prepared once per
device, however many there are."""
import host_program


def test_resident_clusters_go_by_the_launchs_shape(tmp_path):
    out = host_program.run("""
#include <cstdio>
#include "rmsq_ops_plan.h"
int main()
{
    rmsq::ResidentClusters table;
    int kernel[2], asked = 0;
    const auto get = [&](int fn, int dev, unsigned threads, int smem, int cluster, int answer) {
        return table.get({&kernel[fn], dev, threads, smem, cluster}, [&]() { ++asked; return answer; });
    };
    int wrong = get(0, 0, 352, 200000, 16, 7) != 7;
    // another kernel, device, number of threads, ring or cluster is another question
    wrong += get(1, 0, 352, 200000, 16, 6) != 6;
    wrong += get(0, 1, 352, 200000, 16, 5) != 5;
    wrong += get(0, 0, 384, 200000, 16, 4) != 4;
    wrong += get(0, 0, 352, 100000, 16, 14) != 14;
    wrong += get(0, 0, 352, 200000, 8, 18) != 18;
    wrong += asked != 6;
    // and each is asked once
    wrong += get(0, 0, 352, 200000, 16, 99) != 7 || get(0, 0, 352, 100000, 16, 99) != 14 || asked != 6;
    // a failed question is not kept
    wrong += get(0, 0, 64, 0, 2, 0) != 0 || get(0, 0, 64, 0, 2, 60) != 60 || get(0, 0, 64, 0, 2, 99) != 60;
    std::printf("%d\\n", wrong);
}
""", tmp_path)
    assert out.strip() == "0"


def test_more_prepared_kernels_than_any_process_has(tmp_path):
    # 200 kernels on each of 64 devices
    out = host_program.run("""
#include <cstdio>
#include "rmsq_ops_plan.h"
static char kernels[200];
int main()
{
    rmsq::PreparedKernels table;
    int wrong = 0;
    for (int dev = 0; dev < 64; ++dev)
        for (char& k : kernels) {
            wrong += table.has(&k, dev);
            table.add(&k, dev);
        }
    for (int dev = 0; dev < 64; ++dev)
        for (char& k : kernels) wrong += !table.has(&k, dev);
    std::printf("%d\\n", wrong + table.has(kernels, 64));
}
""", tmp_path)
    assert out.strip() == "0"
