// Host-side hooks of the training operators' translation units.
#pragma once

namespace psk {

// The status words (read, then zeroed if `reset`) of the resident loss kernel,
// of the norm backward's ring kernel and of the matrix products, and their
// copies of the lost-copy test hook.
int loss_status(unsigned int* v, bool reset);
int loss_set_drop_row(long long row);
int norm_bwd_status(unsigned int* v, bool reset);
int norm_bwd_set_drop_row(long long row);
int mm_status(unsigned int* v, bool reset);
int ortho_small_status(unsigned int* v, bool reset);
int mm_set_drop_row(long long row);

}  // namespace psk
