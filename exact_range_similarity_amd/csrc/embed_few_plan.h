// How k_embed_grad_few is launched.  Host arithmetic alone, no HIP.
#pragma once

#include <cstdint>

namespace ersj {

constexpr int kFewMax = 1024;  // tokens
constexpr int kFewRows = 64;   // rows of the table to a workgroup, one to a lane
constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / 64;
// A launch holds less than 2^32 work items along an axis; 2^31 are used.
constexpr int64_t kFewGroups = ((int64_t)1 << 31) / kFewThreads;

struct FewPlan {
    int own;       // rows of a workgroup
    int64_t step;  // rows of a launch; tables of more than 2^28 rows take several
};

// As many rows to a workgroup as leave four workgroups to each CU, and no more than kFewRows.
inline FewPlan few_plan(int64_t rows)
{
    const int64_t want = (rows + 1023) / 1024;
    FewPlan p;
    p.own = want < kFewWaves ? kFewWaves : want > kFewRows ? kFewRows : (int)want;
    p.step = kFewGroups * p.own;
    return p;
}

// Workgroups of the launch for the rows from `v`.
inline uint32_t few_groups(const FewPlan &p, int64_t rows, int64_t v)
{
    const int64_t n = rows - v < p.step ? rows - v : p.step;
    return (uint32_t)((n + p.own - 1) / p.own);
}

}  // namespace ersj
