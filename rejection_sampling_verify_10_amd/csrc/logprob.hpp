// Log probabilities of given tokens and their gradient: argument blocks.
#pragma once

#include "common.hpp"
#include "internal.hpp"

namespace sv {

constexpr int kLpThreads = 512;
constexpr int kLpStats = 3;         // floats of a row's statistics: largest logit, log2 of the sum, entropy

struct LogprobArgs {
    const void* logits;             // row r at logits + r*stride elements
    long long stride;
    int dtype, R, V;
    const int32_t* tokens;          // [R][M] (M 0: none)
    int M, top_n;
    float c;                        // log2(e) / T
    float* out_lp;                  // [R][M]
    float* out_entropy;             // [R] or null
    float* out_stats;               // [R][kLpStats] or null
    int32_t* out_top;               // [R][top_n]
    float* out_top_lp;              // [R][top_n]
    int per, slices;                // vectors of a workgroup, workgroups a row
    unsigned long long* words;      // [R][slices][kLpHead + top_n] (slices > 1), zero before and after a call
    unsigned* done;                 // [R] slices that have written theirs, zero before and after a call
};
constexpr int kLpHead = 3;          // words of a slice's record before its list: largest logit, S, W

struct LogprobGradArgs {
    const void* logits;
    void* grad;                     // row r at grad + r*grad_stride elements
    long long stride, grad_stride;
    int dtype, R, V;
    const int32_t* tokens;          // [R][M]
    int M;
    const float* stats;             // [R][kLpStats]
    const float* g_lp;              // [R][M]
    const float* g_entropy;         // [R] or null
    float c, invT;
    int slices;                     // workgroups a row
};

// Fills per and slices.
void logprob_plan(LogprobArgs& a);
hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s, Timing t = {});
hipError_t launch_logprobs_grad(const LogprobGradArgs& a, hipStream_t s, Timing t = {});
int logprob_grad_slices(int dtype, int V);

}  // namespace sv
