// Launch function of the sampler (kie_sample.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

struct SampleArgs {
    const void* logits;          // [rows][vocab], row_stride elements apart
    int32_t type;                // 0 fp16, 1 bf16, 2 fp32
    int32_t rows, vocab;
    int64_t row_stride;
    const float* temperature;    // [rows] or null: 1
    const int32_t* top_k;        // [rows] or null: off
    const float* top_p;          // [rows] or null: off
    const float* min_p;          // [rows] or null: off
    const float* u;              // [rows]
    int32_t* tokens;             // [rows]
    float* probs;                // [rows] or null
    int32_t* next;               // [rows] or null: the tokens again, 0 for -1 (an engine's next input)
};

// Largest vocabulary: row sums of 44-bit weights stay below 2^62.
#define KIE_SAMPLE_MAX_VOCAB (1 << 18)

extern "C" cudaError_t kie_launch_sample(const SampleArgs* a, int sms, cudaStream_t st);
