// token_rules.h -- settings of the losses over given tokens: dlm_policy_params and
// dlm_preference_params as the kernels use them.
#pragma once

namespace dlm {

struct PolicyRule {
    float lo, hi;     // 1 - clip_low, 1 + clip_high
    float dual;       // 0: none
    float kl_weight;
    int kl;           // DLM_KL_*
};

struct PreferenceRule {
    double beta;
    float smooth;     // label smoothing
    int kind;         // DLM_PREF_*
};

}  // namespace dlm
