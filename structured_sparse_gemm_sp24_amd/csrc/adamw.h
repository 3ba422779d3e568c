// Host side of the AdamW step (internal to the library): what a launch takes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sp24 {

struct AdamTensor {
    const float* p;
    float* p_out;
    const char *g, *m;
    char* m_out;
    const char* v;
    char* v_out;
    const uint8_t* ms;
    uint8_t* ms_out;
    const uint8_t* vs;
    uint8_t* vs_out;
    char* copy;
    int64_t n;
    uint32_t index;
};

// What changes from step to step.
struct AdamScalars {
    float decay, rate, root;  // 1 - lr weight_decay, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
    uint32_t key;             // of seed and t
};

constexpr int ADAM_TENSORS = 32, ADAM_CHUNK = 2048;  // tensors a launch, elements a workgroup

struct AdamArgs {
    AdamTensor t[ADAM_TENSORS];
    uint32_t first[ADAM_TENSORS];  // first workgroup of each
    AdamScalars now;
    const AdamScalars* later;  // in their place where not NULL
    const float* grad_scale;
    float b1, c1, b2, c2, eps;
    int count;
};
static_assert(sizeof(AdamArgs) <= 4096, "a kernel's arguments");

struct AdamSchedule {
    double lr, beta1, beta2, decay;
    const float* lr_dev;
    const int64_t* step_dev;
    int64_t step;
    uint64_t seed;
};

AdamScalars adam_scalars(const AdamSchedule& h);  // from lr and step
hipError_t launch_adam_scalars(const AdamSchedule& h, AdamScalars* out, hipStream_t s);
// grad, copy: 0 bf16, 1 fp16, 2 fp32.
hipError_t launch_adamw(const AdamArgs& a, int grad, bool bits8, int copy, unsigned blocks, hipStream_t s);

}  // namespace sp24
