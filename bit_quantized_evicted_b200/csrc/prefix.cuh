// What the shared-prefix kernel (prefix.cu) leaves for the decode kernel that
// merges it (decode.cu): partial softmax states of the prefix.
#pragma once
#include "common.cuh"

namespace minikv {

constexpr int kPreStride = 132;   // floats of a row's partial: y[128], m, l (m in log2 units)

// The rows of KV head kvh are its query heads of the sharing sequences, in
// order: row = (place among the sharing sequences) * g + head of the group.
// They are cut into tiles of N = 1 << lgN rows; unit u = row tile * Hkv + kvh.
// The units' token tiles (tpu each, T = units * tpu in all) lie end to end and
// are cut into P equal ranges, one a CTA; CTA c writes its state of unit u to
// slot c + u (a range walks c and u upwards together, so no two meet there).
struct PreTab {
    const float *part;   // [P + units][N][kPreStride]
    int lgN, tpu, P, T;
    int listed;          // 1: place[b] holds, 0: every sequence shares
    short place[MINIKV_MAX_RAGGED_SEQS];   // -1: sequence b does not share
};
// sequence b's place among the sharing ones, -1: it attends to nothing of the prefix
__device__ __forceinline__ int prefix_place(const PreTab &t, int b) {
    return t.P == 0 ? -1 : t.listed ? t.place[b] : b;
}
// the CTA whose range [c T / P, (c + 1) T / P) holds tile x
__host__ __device__ __forceinline__ int pre_cta(const PreTab &t, int x) {
    return (int)((((unsigned long long)x + 1) * (unsigned)t.P - 1) / (unsigned)t.T);
}

// A step behind a shared prefix, for decode_launch: once its own checks have
// passed, it queues the prefix pass (prefix_launch) with these before its kernel.
struct PrefixCall {
    const minikv_cache *prefix;
    const int *shared;   // host flags, or NULL: all
    void *ws;            // prefix_workspace_bytes
};

// Queue the prefix pass: states of the sharing sequences' rows over p, and *tab
// for the merging decode kernel (tab->P = 0: nobody attends to anything; nothing
// but a clearing of the status words is queued).
int prefix_launch(const PrefixCall &call, int B, const uint16_t *q, int Hq, float sm_scale, cudaStream_t stream,
                  PreTab *tab);

}  // namespace minikv
