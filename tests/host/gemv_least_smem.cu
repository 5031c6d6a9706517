// The least shared memory that the M <= 8 GEMV asks for with CTAs in clusters,
// over every split of every shape up to 40 row tiles by 64 column groups (larger
// ones need more).  Prints "least=<bytes>".
#include "../../nested_bit_weight_b200/csrc/mq_gemv_tc.cu"

#include <cstdio>

extern "C" size_t mq_plane_bytes(int64_t, int64_t, int) { return 0; }
namespace mq {
mq_status cuda_fail(cudaError_t, const char *) { return MQ_ERR_CUDA; }
void set_error(mq_status, const char *, ...) {}
}  // namespace mq

using namespace mq;

int main() {
    size_t least = (size_t)1 << 30;
    for (long T = 1; T <= 40; ++T)
        for (long G = 1; G <= 64; ++G)
            for (int M = 1; M <= 8; ++M)
                for (int r = 1; r <= 8; ++r)
                    for (int cs = 2; cs <= 8; ++cs) {
                        const long nc = 148 / cs < T ? 148 / cs : T;
                        if (nc < 1 || T / nc * G < cs) continue;
                        const Plan p = plan_for(Work{T, G, (int)nc, cs}, M, r);
                        if (p.ok && p.smem < least) least = p.smem;
                    }
    printf("least=%zu\n", least);
    return 0;
}
