// Host-side hooks of the training operators' translation units.
#pragma once

namespace psk {

// The status words (read, then zeroed if `reset`) of the resident loss kernel
// and of the norm backward's ring kernel, and their copies of the lost-copy
// test hook.
int loss_status(unsigned int* v, bool reset);
int loss_set_drop_row(long long row);
int norm_bwd_status(unsigned int* v, bool reset);
int norm_bwd_set_drop_row(long long row);

}  // namespace psk
