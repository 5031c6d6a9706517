// bind_device (mq_api.cu) against a runtime of two devices that exists only here:
// a stream answers for its device except while it captures.
#include <cuda_runtime.h>
#include <stdio.h>

static int g_current = 0, g_context = 0, g_asked = 0;
static bool g_capturing = false;

static int stream_device(cudaStream_t st) { return (int)(((size_t)st) & 1); }
static cudaError_t fake_is_capturing(cudaStream_t, cudaStreamCaptureStatus *c) {
    *c = g_capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
static cudaError_t fake_stream_device(cudaStream_t st, int *dev) {
    ++g_asked;
    if (g_capturing) return cudaErrorStreamCaptureUnsupported;
    *dev = stream_device(st);
    return cudaSuccess;
}
static cudaError_t fake_get_device(int *dev) { *dev = g_current; return cudaSuccess; }
static cudaError_t fake_set_device(int dev) { g_current = g_context = dev; return cudaSuccess; }
static int fake_ctx(void **p) { *p = &g_context; return 0; }
static int fake_ctx_device(int *dev) { *dev = g_context; return 0; }
static cudaError_t fake_entry(const char *name, void **p, unsigned long long, cudaDriverEntryPointQueryResult *) {
    *p = name[5] == 'G' && name[8] == 'C' ? (void *)fake_ctx : (void *)fake_ctx_device;
    return cudaSuccess;
}
static cudaError_t fake_sync() { return cudaSuccess; }

#define cudaStreamIsCapturing fake_is_capturing
#define cudaStreamGetDevice fake_stream_device
#define cudaGetDevice fake_get_device
#define cudaSetDevice fake_set_device
#define cudaGetDriverEntryPoint fake_entry
#define cudaDeviceSynchronize fake_sync
#include "mq_api.cu"

// what mq_api.cu calls beside
namespace mq {
bool gemv_tc_supported(int64_t, int64_t, int64_t, int) { return false; }
size_t gemv_tc_workspace_bytes(int64_t, int64_t, int64_t, int) { return 0; }
size_t gemm_tc_workspace_bytes(int64_t, int64_t, int64_t, int) { return 0; }
mq_status launch_gemv_tc(const uint16_t *, const mq_weights *, int64_t, uint16_t *, void *, size_t, cudaStream_t) { return MQ_OK; }
mq_status launch_gemm_tc(const uint16_t *, const mq_weights *, int64_t, uint16_t *, void *, size_t, cudaStream_t) { return MQ_OK; }
bool gemv_tc_take_timeout(bool *) { return true; }
bool gemm_tc_take_timeout(bool *) { return true; }
bool mx4_take_timeout(bool *) { return true; }
}  // namespace mq

static int g_bad = 0, g_checked = 0;
static void expect(cudaStream_t st, int want, const char *what) {
    ++g_checked;
    if (mq::bind_device(st) != MQ_OK || g_current != want) {
        ++g_bad;
        printf("%s: device %d, expected %d\n", what, g_current, want);
    }
}

int main() {
    cudaStream_t s0 = (cudaStream_t)0x1000, s1 = (cudaStream_t)0x2001, t1 = (cudaStream_t)0x3001;
    expect(s1, 1, "a stream's own device");
    expect(s0, 0, "another stream's device");
    expect(s1, 1, "and back");
    // the caller moves to another device and comes back with the same stream
    fake_set_device(0);
    expect(s1, 1, "the same stream from another device");
    // a first call within a capture goes to the caller's device, the next outside it to the stream's
    fake_set_device(0);
    g_capturing = true;
    expect(t1, 0, "a capturing stream: the caller's device");
    g_capturing = false;
    expect(t1, 1, "the same stream after the capture");
    // a remembered stream is not asked again, nor while it captures
    const int asked = g_asked;
    expect(t1, 1, "remembered");
    g_capturing = true;
    fake_set_device(1);
    expect(t1, 1, "remembered, capturing");
    g_capturing = false;
    ++g_checked;
    if (g_asked != asked) { ++g_bad; printf("a remembered stream was asked for its device\n"); }
    // the legacy stream: the caller's device
    fake_set_device(0);
    expect(nullptr, 0, "legacy stream");
    expect(t1, 1, "a stream after the legacy one");
    printf("checked=%d bad=%d\n", g_checked, g_bad);
    return g_bad != 0;
}
