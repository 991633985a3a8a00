// Which of a call's rules on scores are in use. Plain C++, so that the CPU tests run the same code.
#pragma once

#include "simcomm.h"

namespace simcomm {

// The rules without the arrays of a rule that is left out. A caller may leave anything in those: they are neither
// checked nor read.
inline coll_logit_rules_t rules_in_use(coll_logit_rules_t u) {
    if (!u.history_len) {
        u.history = u.prompt_len = nullptr;
        u.repetition = u.frequency = u.presence = nullptr;
        u.ld_history = 0;
    }
    if (!u.bias_start) {
        u.bias_token = nullptr;
        u.bias_value = nullptr;
        u.bias_count = 0;
    }
    if (!u.mask) {
        u.mask_row = nullptr;
        u.ld_mask = u.mask_rows = 0;
    }
    return u;
}

}  // namespace simcomm
